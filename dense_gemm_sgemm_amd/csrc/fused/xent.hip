// Softmax cross entropy of X * W^T without storing the logits, and its
// gradients: C entry points, the join of the tiles' softmax statistics, and
// the preparations of the backward pass.
#define MI355FUSED_BUILDING 1
#include "fused.hpp"

namespace mi355gemm {
namespace fused {
namespace {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
constexpr int kPrepareThreads = 256;

// ---- The join.  The kLse tiles leave, for each row, a maximum t_c and a sum
// of exp(z - t_c) for each chunk c of the columns.  With t = max t_c:
// lse = t + log(sum_c s_c exp(t_c - t)).  A workgroup of 16 waves takes 16
// rows; the four groups of 16 lanes of its waves share the chunks 64 ways,
// eight loads in flight each.
constexpr int kJoinWaves = 16, kJoinRows = 16, kJoinParts = 4 * kJoinWaves;

struct JoinArgs {
  const float2* partial;
  const float* target_logit;
  const long long* targets;
  long long ignore, vocab;
  float *loss, *lse;
  int64_t ld;
  int M, chunks;
};

__device__ __forceinline__ void join(float& t, float& s, float t2, float s2) {
  const float top = fmaxf(t, t2);
  const float base = fabsf(top) == __builtin_inff() ? 0.f : top;   // (0 * exp(-inf), inf)
  s = s * __expf(t - base) + s2 * __expf(t2 - base);
  t = top;
}

__global__ __launch_bounds__(64 * kJoinWaves) void join_kernel(JoinArgs p, int64_t base) {
  __shared__ float2 part[kJoinParts][kJoinRows];
  const int row = threadIdx.x & 15, mine = threadIdx.x >> 4;
  const int64_t m = (base + blockIdx.x) * kJoinRows + row;
  float t = -__builtin_inff(), s = 0.f;
  if (m < p.M) {
    constexpr int U = 8;   // chunks in flight
    for (int c = mine; c < p.chunks; c += U * kJoinParts) {
      float2 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int cu = c + u * kJoinParts;
        v[u] = cu < p.chunks ? p.partial[cu * p.ld + m] : make_float2(-__builtin_inff(), 0.f);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) join(t, s, v[u].x, v[u].y);
    }
  }
  part[mine][row] = make_float2(t, s);
  __syncthreads();
  // halving over the parts, in a fixed order
  for (int half = kJoinParts / 2; half >= 1; half /= 2) {
    if (mine < half) {
      const float2 o = part[mine + half][row];
      join(t, s, o.x, o.y);
      part[mine][row] = make_float2(t, s);
    }
    __syncthreads();
  }
  if (mine != 0 || m >= p.M) return;
  const float lse = t + __logf(s);
  const long long y = p.targets[m];
  float loss = 0.f;
  if (y != p.ignore)
    loss = y >= 0 && y < p.vocab ? lse - p.target_logit[m] : __builtin_nanf("");
  p.lse[m] = lse;
  p.loss[m] = loss;
}

// ---- The scale of d: {f, 1 / f} with f = size / max |dloss| over the rows that
// count and are finite, so that d = (p - [target]) dloss f has its largest
// entries at `size`.  With one dloss for all rows (a mean) they are p - 1 times
// `size`, a power of two: rounding dloss itself to 16 bits, the same way in
// every row, would put all gradients off by up to 2^-9 in bf16 (measured: 0.34 %
// against 0.17 % of random rounding).  In fp16 the size 2^14 also keeps
// probabilities down to 2^-38 (binary16's smallest step is 2^-24).  1 where that
// maximum is 0.
struct ScaleArgs {
  const float* dloss;
  const long long* targets;
  long long ignore;
  float* scale;
  float size;
  int M;
};

__device__ __forceinline__ void find_scale(const ScaleArgs& p) {
  __shared__ float part[kPrepareThreads / 64];
  float top = 0.f;
  for (int m = threadIdx.x; m < p.M; m += kPrepareThreads) {
    const float v = fabsf(p.dloss[m]);
    if (p.targets[m] != p.ignore && v < __builtin_inff()) top = fmaxf(top, v);
  }
#pragma unroll
  for (int k = 32; k >= 1; k /= 2) top = fmaxf(top, __shfl_xor(top, k));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < kPrepareThreads / 64; ++w) top = fmaxf(top, part[w]);
  float f = 1.f, r = 1.f;
  if (top > 0.f) {
    top = fmaxf(top, 0x1p-100f);   // f stays finite
    f = p.size / top;
    r = top / p.size;
  }
  p.scale[0] = f;
  p.scale[1] = r;
}

// What the backward pass needs first, in one launch: the last workgroup finds
// the scale of d, the others transpose X and clear the rows of d that no
// tile writes.
struct PrepareArgs {
  Transpose x;
  half_t* zero;
  int64_t zero_pieces;      // of 16 bytes
  int64_t blocks_x, blocks_zero;
  ScaleArgs scale;
};

__global__ __launch_bounds__(kPrepareThreads) void prepare_kernel(PrepareArgs p, int64_t base) {
  const int64_t b = base + blockIdx.x;
  if (b < p.blocks_x) {
    transpose_tile(p.x, b * (kPrepareThreads / 64) + (threadIdx.x >> 6), threadIdx.x & 63);
  } else if (b < p.blocks_x + p.blocks_zero) {
    const int64_t t = (b - p.blocks_x) * kPrepareThreads + threadIdx.x;
    if (t < p.zero_pieces) *((h8*)p.zero + t) = h8{};
  } else {
    find_scale(p.scale);
  }
}

int check(int type, int M, int N, int K) {
  const int status = check_sizes(M, N, K);
  if (status != GEMM_OK) return status;
  return bad_type(type) || (N == 0 && M > 0) ? GEMM_ERR_BAD_ARG : GEMM_OK;
}

const half_t* in16(const void* p) { return static_cast<const half_t*>(p); }
half_t* out16(void* p) { return static_cast<half_t*>(p); }

// ---- Pieces of the columns.  A piece's d ([rows][width], 16-bit) takes about
// kPieceBytes at most, so that it is written and read twice mostly out of the
// last-level cache; pieces are at least 2048 wide, which keeps the products'
// K deep, and a multiple of 256.  The last one starts early enough to be 128
// wide; its columns that the one before has had are zero in d.
constexpr size_t kPieceBytes = size_t(256) << 20;
constexpr int kMinPiece = 2048;

struct BwdPlan {
  int Mp, Ms, Np, Kp;     // Ms: whole slabs of rows (they are summed over for dW)
  int width, pieces;      // every piece but the last is `width` columns
  int64_t ldd;            // leading dimension of a piece's d
  GradXPlan gx;           // for `width` columns
  size_t bytes_d, bytes_tail, bytes_sum = 0, bytes_scale, bytes_xt, bytes_x = 0, bytes_w = 0;
  size_t total() const {
    return bytes_d + bytes_tail + bytes_sum + bytes_scale + bytes_xt + bytes_x + bytes_w;
  }
};
BwdPlan plan_bwd(int M, int N, int K, Mat X, Mat W, bool dx, bool dw) {
  BwdPlan p;
  p.Mp = pad_rows(M);
  p.Ms = pad_slabs(M);
  p.Np = pad_rows(N);
  p.Kp = pad_k(K);
  const int64_t most = std::max<int64_t>(kMinPiece, kPieceBytes / ((size_t)p.Mp * 2) / 256 * 256);
  const int64_t n = (p.Np + most - 1) / most;
  p.width = (int)std::min<int64_t>(round_up((p.Np + n - 1) / n, 256), p.Np);
  p.pieces = (p.Np + p.width - 1) / p.width;
  p.ldd = round_up(std::max(p.width, 128), 64);
  p.bytes_d = round256((size_t)p.Ms * p.ldd * 2);
  p.bytes_tail = dx ? (size_t)p.Mp * 128 : 0;
  if (dx) {
    p.gx = plan_grad_x(p.Mp, p.Kp, (p.width + 63) / 64, p.pieces > 1);
    if (p.pieces > 1 || p.gx.splits > 1)
      p.bytes_sum = round256((size_t)p.gx.splits * p.Mp * p.Kp * sizeof(float));
  }
  p.bytes_scale = 256;
  p.bytes_xt = dw ? round256((size_t)p.Kp * p.Ms * 2) : 0;
  // (M == 0: dW = 0, X and W are not read and may be null)
  if (M > 0 && needs_copy(X.p, X.ld, M, K)) p.bytes_x = copy_bytes(M, K);
  if (M > 0 && needs_copy(W.p, W.ld, N, K)) p.bytes_w = copy_bytes(N, K);
  return p;
}

}  // namespace
}  // namespace fused
}  // namespace mi355gemm

using namespace mi355gemm;
using namespace mi355gemm::fused;

extern "C" {

MI355FUSED_API unsigned long long gemm_xent_workspace(int type, int M, int N, int K, const void* X,
                                                      int ldx, const void* W, int ldw) {
  if (check(type, M, N, K) != GEMM_OK || M == 0 || bad_ld(ldx, K) || bad_ld(ldw, K)) return 0;
  return round256((size_t)lse_chunks(M, N, K) * M * sizeof(float2)) + round256((size_t)M * sizeof(float)) +
         (needs_copy(X, ldx, M, K) ? copy_bytes(M, K) : 0) +
         (needs_copy(W, ldw, N, K) ? copy_bytes(N, K) : 0);
}

MI355FUSED_API int gemm_xent(int type, int M, int N, int K, const void* X, int ldx, const void* W,
                             int ldw, const long long* targets, long long ignore, float* loss,
                             float* lse, void* workspace, unsigned long long workspace_bytes,
                             void* stream) {
  const int status = check(type, M, N, K);
  if (status != GEMM_OK) return status;
  if (M == 0) return GEMM_OK;
  if (bad_ld(ldx, K) || bad_ld(ldw, K)) return GEMM_ERR_BAD_LD;
  if (targets == nullptr || loss == nullptr || lse == nullptr ||
      (K > 0 && (X == nullptr || W == nullptr)))
    return GEMM_ERR_NULL_POINTER;
  const size_t need = gemm_xent_workspace(type, M, N, K, X, ldx, W, ldw);
  if (!workspace_ok(need, workspace, workspace_bytes)) return GEMM_ERR_WORKSPACE;
  const int cus = check_device();
  if (cus < 0) return cus;
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  float2* partial = reinterpret_cast<float2*>(ws);
  ws += round256((size_t)lse_chunks(M, N, K) * M * sizeof(float2));
  float* target_logit = reinterpret_cast<float*>(ws);
  ws += round256((size_t)M * sizeof(float));
  PadJobs jobs;
  const Mat x = jobs.add(Mat{in16(X), ldx}, M, K, ws);
  const Mat w = jobs.add(Mat{in16(W), ldw}, N, K, ws);
  hipError_t e = launch_pad(jobs, s);
  if (e != hipSuccess) return to_status(e);
  Args16 a{x.p, w.p, nullptr, x.ld, w.ld, 0, pad_rows(M), pad_rows(N), pad_k(K)};
  a.fmt = type == GEMM_TYPE_BF16 ? kFmtBF16 : kFmtF16;
  FusedExtra f;
  f.m_end = M;
  f.n_end = N;
  f.targets = targets;
  f.ignore = ignore;
  f.target_logit = target_logit;
  f.partial = partial;
  f.ld_partial = M;
  e = launch_lse_tiles(a, f, cus, s);
  if (e != hipSuccess) return to_status(e);
  const JoinArgs j{partial, target_logit, targets, ignore, N, loss, lse, M, M,
                   lse_chunks(M, N, K)};
  return to_status(launch_tiles((const void*)join_kernel, j,
                                ((int64_t)M + kJoinRows - 1) / kJoinRows, 64 * kJoinWaves, 0, s));
}

MI355FUSED_API unsigned long long gemm_xent_bwd_workspace(int type, int M, int N, int K,
                                                          const void* X, int ldx, const void* W,
                                                          int ldw, int want_dx, int want_dw) {
  if (check(type, M, N, K) != GEMM_OK || K == 0 || N == 0 || bad_ld(ldx, K) || bad_ld(ldw, K))
    return 0;
  const bool dx = want_dx && M > 0;
  if (!dx && !want_dw) return 0;
  return plan_bwd(M, N, K, Mat{in16(X), ldx}, Mat{in16(W), ldw}, dx, want_dw != 0).total();
}

MI355FUSED_API int gemm_xent_bwd(int type, int M, int N, int K, const void* X, int ldx,
                                 const void* W, int ldw, const long long* targets,
                                 long long ignore, const float* lse, const float* dloss, void* dX,
                                 int lddx, void* dW, int lddw, void* workspace,
                                 unsigned long long workspace_bytes, void* stream) {
  const int status = check(type, M, N, K);
  if (status != GEMM_OK) return status;
  const bool dx = dX != nullptr && M > 0 && K > 0;
  const bool dw = dW != nullptr && N > 0 && K > 0;
  if (!dx && !dw) return GEMM_OK;
  if (bad_ld(ldx, K) || bad_ld(ldw, K) || (dx && bad_ld(lddx, K)) || (dw && bad_ld(lddw, K)))
    return GEMM_ERR_BAD_LD;
  if (M > 0 && (X == nullptr || W == nullptr || targets == nullptr || lse == nullptr ||
                dloss == nullptr))
    return GEMM_ERR_NULL_POINTER;
  const BwdPlan p = plan_bwd(M, N, K, Mat{in16(X), ldx}, Mat{in16(W), ldw}, dx, dw);
  if (!workspace_ok(p.total(), workspace, workspace_bytes)) return GEMM_ERR_WORKSPACE;
  const int cus = check_device();
  if (cus < 0) return cus;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int fmt = type == GEMM_TYPE_BF16 ? kFmtBF16 : kFmtF16;
  char* ws = static_cast<char*>(workspace);
  half_t* d = reinterpret_cast<half_t*>(ws);
  ws += p.bytes_d;
  half_t* tail = reinterpret_cast<half_t*>(ws);
  ws += p.bytes_tail;
  float* sum = reinterpret_cast<float*>(ws);
  ws += p.bytes_sum;
  float* scale = reinterpret_cast<float*>(ws);
  ws += p.bytes_scale;
  half_t* xt = reinterpret_cast<half_t*>(ws);
  ws += p.bytes_xt;
  PadJobs jobs;
  Mat x{in16(X), ldx}, w{in16(W), ldw};
  if (p.bytes_x) x = jobs.copy(x, M, K, ws);
  if (p.bytes_w) w = jobs.copy(w, N, K, ws);
  hipError_t e = launch_pad(jobs, s);
  if (e != hipSuccess) return to_status(e);
  PrepareArgs prep{};
  if (dw) {
    prep.x = Transpose{in16(X), xt, ldx, p.Ms, M, K, p.Ms, p.Kp, targets, ignore};
    prep.blocks_x = (prep.x.tiles() + kPrepareThreads / 64 - 1) / (kPrepareThreads / 64);
    // the rows of d that no piece writes (all of them for M == 0) are zero
    const int64_t written = M > 0 ? p.Mp : 0;
    prep.zero = d + written * p.ldd;
    prep.zero_pieces = (p.Ms - written) * p.ldd / 8;
    prep.blocks_zero = (prep.zero_pieces + kPrepareThreads - 1) / kPrepareThreads;
  }
  prep.scale = ScaleArgs{dloss, targets, ignore, scale, fmt == kFmtF16 ? 0x1p14f : 1.f, M};
  e = launch_tiles((const void*)prepare_kernel, prep, prep.blocks_x + prep.blocks_zero + 1,
                   kPrepareThreads, 0, s);
  if (e != hipSuccess) return to_status(e);
  for (int i = 0; i < p.pieces; ++i) {
    const bool last = i + 1 == p.pieces;
    const int owned = i * p.width;   // first column that this piece stores
    const int end = last ? p.Np : owned + p.width;
    const int begin = std::min(owned, end - 128);
    const int width = end - begin;
    const half_t* wp = w.p + (int64_t)begin * w.ld;
    // d of the piece
    Args16 a{x.p, wp, d, x.ld, w.ld, p.ldd, p.Mp, width, p.Kp};
    a.fmt = fmt;
    FusedExtra f;
    f.m_end = M;
    f.n_begin = owned - begin;
    f.n_end = N - begin;
    f.targets = targets;
    f.ignore = ignore;
    f.vocab = N;
    f.col0 = begin;
    f.lse = lse;
    f.row_scale = dloss;
    f.scale = scale;
    f.tail = dx && width % 64 != 0 ? tail : nullptr;
    f.ldt = 64;
    if (M > 0) e = launch_dlogit_tiles(a, f, cus, s);
    if (e != hipSuccess) return to_status(e);
    if (dw) {
      Args16 b{d, xt, out16(dW) + (int64_t)begin * lddw, p.ldd, p.Ms, lddw,
               (int)round_up(width, 8), p.Kp, p.Ms};
      b.fmt = fmt;
      FusedExtra g;
      g.m_begin = owned - begin;
      g.m_end = N - begin < width ? N - begin : width;
      g.n_end = K;
      g.scale = scale;
      e = launch_grad_w(b, g, cus, s);
      if (e != hipSuccess) return to_status(e);
    }
    if (dx) {
      Args16 b{d, wp, out16(dX), p.ldd, w.ld, lddx, p.Mp, p.Kp, width};
      b.fmt = fmt;
      FusedExtra g;
      g.m_end = M;
      g.n_end = K;
      g.tail = f.tail;
      g.ldt = 64;
      g.scale = scale;
      // (the last piece has fewer columns: fewer slabs a range, not fewer ranges)
      GradXPlan plan = p.gx;
      const int slabs = (width + 63) / 64;
      if (last && p.pieces > 1) {
        plan.per = (slabs + plan.splits - 1) / plan.splits;
        plan.splits = (slabs + plan.per - 1) / plan.per;
      }
      if (p.bytes_sum) {
        g.sum = sum;
        g.ld_sum = p.Kp;
        g.split_stride = (int64_t)p.Mp * p.Kp;
        g.sum_add = i > 0;
      }
      e = launch_grad_x(b, g, plan, cus, s);
      if (e == hipSuccess && last && g.sum)
        e = launch_sums(fmt, g, p.gx.splits, out16(dX), lddx, M, K, s);
      if (e != hipSuccess) return to_status(e);
    }
  }
  return GEMM_OK;
}

}  // extern "C"

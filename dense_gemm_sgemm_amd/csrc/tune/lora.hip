// Low-rank adapters beside a shared projection, and their gradients: C entry
// points.
#define MI355TUNE_BUILDING 1
#include "tune.hpp"

namespace mi355gemm {
namespace tune {
namespace {

using fused::bad_ld;
using fused::copy_bytes;
using fused::kMinRows;
using fused::line_ld;
using fused::needs_copy;
using fused::pad_k;
using fused::pad_rows;
using fused::PadJobs;

const half_t* in16(const void* p) { return static_cast<const half_t*>(p); }
half_t* out16(void* p) { return static_cast<half_t*>(p); }

int check(int type, int M, int N, int K, int R, int S) {
  if (R < 0 || S < 0) return GEMM_ERR_NEGATIVE_DIM;
  const int status = fused::check_sizes(M, N, K);
  if (status != GEMM_OK) return status;
  return fused::bad_type(type) || R < 1 || R > kMaxRank || S > fused::kMaxSize ? GEMM_ERR_BAD_ARG
                                                                              : GEMM_OK;
}

// Rows in blocks of 64 times columns: what the kernels for few rows (lora_rows.hip,
// lora_dx.hip) take their time for; the tiles' is the same up to 256 of them.
int64_t row_work(int M, int cols) { return ((int64_t)M + 63) / 64 * cols; }

// Forward: the kernel for few rows streams W once for 64 of them.  bf16, K and N of
// 4096, M = 128: 30 us against 45 of the tiles, 192: 43 against 44, 256: 56 against
// 44; N 8192, K 2048, M = 96: 38 against 33.  Odd widths cost it more and the tiles
// their copies: N 2305, K 769, M = 192: 20 against 24, 256: 29 against 24.
bool by_rows(int M, int N, Mat x, Mat w) {
  auto even = [](Mat m) { return m.ld % 2 == 0 && (reinterpret_cast<uintptr_t>(m.p) & 3) == 0; };
  return M <= 64 || row_work(M, N) <= (even(x) && even(w) ? 12288 : 8192);
}
// dX = dC W: its kernel for few rows cuts N, the sum's length, which the tiles walk
// whole, but writes and reads its ranges' sums.  bf16, 16 ranks, N 4096 and K 4096, M =
// 192: 42 us against 45, 256: 40 against 44 (64 ranks: 61 against 52), 320: 47 against
// 45; N 6000, K 768, M = 1000: 46 against 75; N 8192, K 2048, M = 640: 62 against 78; N
// 8000, K 512, M = 3000: 89 against 78; N 3000, K 768, M = 1500: 47 against 46; N 1024,
// K 4096, M = 96: 20 against 18; N 2305, K 769, M = 448: 39 against 41.  (It does not
// look at the ranks: with 64 of them the tiles are the faster ones from 256 rows on.)
bool dx_by_rows(int M, int N, int K) {
  return M <= 64 || row_work(M, K) <= std::min<int64_t>(4 * (int64_t)N - 2000, 24000);
}

struct Plan {
  size_t t2, factor, x = 0, w = 0, b = 0;
  size_t total() const { return t2 + factor + x + w + b; }
};
Plan make_plan(int M, int N, int K, int R, int S, Mat x, Mat w, int ldb) {
  Plan p;
  p.t2 = round256((size_t)M * rank_ld2(R) * 2);
  p.factor = round256((size_t)M * rank_blocks(R) * sizeof(float));
  if (N > 0 && !by_rows(M, N, x, w)) {
    if (needs_copy(x.p, x.ld, M, K)) p.x = copy_bytes(M, K);
    if (needs_copy(w.p, w.ld, N, K)) p.w = copy_bytes(N, K);
    // (the tiles read B's ranks eight at a time, at 32-bit offsets)
    if (R % 8 != 0 || ldb >= 1 << 22) p.b = round256((size_t)S * N * 16 * rank_blocks(R) * 2);
  }
  return p;
}

// The workspace of the backward pass: t2 and factor of dt, dt itself, both
// stacks of factors turned, the rows by adapter, dt and t packed, their steps'
// factors, partial sums; padded copies of dC and W.
struct BwdPlan {
  bool dx, da, db, few = false;   // few: dX by the kernel for few rows
  DxPlan sums;
  size_t t2 = 0, factor = 0, dt = 0, at = 0, bt = 0;
  size_t first = 0, rows = 0, steps = 0, pack = 0, step_factor = 0, partial[2] = {0, 0};
  size_t copy_c = 0, copy_w = 0, tail = 0;
  GradPlan grad{};
  size_t total() const {
    return t2 + factor + dt + at + bt + first + rows + steps + 2 * pack + 2 * step_factor +
           partial[0] + partial[1] + copy_c + copy_w + tail +
           sums.bytes;
  }
};
size_t copy_bytes_w(int N, int K) {
  return round256((size_t)pad_k(pad_rows(N)) * line_ld(pad_k(K)) * 2);
}
BwdPlan plan_bwd(int M, int N, int K, int R, int S, Mat c, Mat w, bool dx, bool da, bool db) {
  BwdPlan p;
  p.dx = dx && M > 0 && K > 0;
  p.da = da && S > 0 && K > 0;
  p.db = db && S > 0 && N > 0;
  if (M > 0 && S > 0 && (p.dx || p.da)) {
    p.bt = round256((size_t)S * R * line_ld(round_up(N, 8)) * 2);
    if (p.da) p.dt = round256((size_t)M * R * sizeof(float));
  }
  if (p.dx) {
    p.t2 = round256((size_t)M * rank_ld2(R) * 2);
    p.factor = round256((size_t)M * rank_blocks(R) * sizeof(float));
    p.at = round256((size_t)S * K * 16 * rank_blocks(R) * 2);
    p.few = dx_by_rows(M, N, K);
    if (p.few) {
      p.sums = plan_dx(M, N, K);
    } else {
      const int Kd = pad_k(N);
      if (needs_copy(c.p, c.ld, M, N)) p.copy_c = copy_bytes(M, N);
      if (needs_copy(w.p, w.ld, N, K) || Kd != N) p.copy_w = copy_bytes_w(N, K);
      if (Kd % 64 != 0) p.tail = (size_t)pad_rows(M) * 64 * 2;
    }
  }
  if (p.da || p.db) {
    // (the same whatever is asked for, so that each gradient has the same bits)
    p.grad = plan_grad(M, N, K, R, S);
    p.first = round256(((size_t)S + 1) * sizeof(int));
    p.rows = round256((size_t)p.grad.steps * 32 * sizeof(int));
    p.steps = round256((size_t)p.grad.steps * sizeof(int));
    p.pack = p.grad.pack;
    p.step_factor = round256((size_t)p.grad.steps * sizeof(float));
    if (p.da) p.partial[0] = p.grad.partial[0];
    if (p.db) p.partial[1] = p.grad.partial[1];
  }
  return p;
}

// A stack of S matrices: matrices may be any distance apart.
bool bad_stride(long long stride, int S) { return S > 1 && stride < 0; }
// ... which must not overlap where they are written.
bool bad_out_stride(long long stride, int S, int64_t rows, int64_t ld, int64_t cols) {
  return S > 1 && stride < (rows - 1) * ld + cols;
}

}  // namespace
}  // namespace tune
}  // namespace mi355gemm

using namespace mi355gemm;
using namespace mi355gemm::tune;

extern "C" {

MI355TUNE_API unsigned long long gemm_lora_workspace(int type, int M, int N, int K, int R, int S,
                                                     const void* X, int ldx, const void* W,
                                                     int ldw, int ldb) {
  if (check(type, M, N, K, R, S) != GEMM_OK || M == 0 || bad_ld(ldx, K) ||
      (N > 0 && bad_ld(ldw, K)))
    return 0;
  return make_plan(M, N, K, R, S, Mat{in16(X), ldx}, Mat{in16(W), ldw}, ldb).total();
}

MI355TUNE_API int gemm_lora(int type, int M, int N, int K, int R, int S, const void* X, int ldx,
                            const void* W, int ldw, const void* A, int lda, long long stride_a,
                            const void* B, int ldb, long long stride_b, const long long* ids,
                            const float* scales, const void* bias, int act, const void* residual,
                            int ldr, void* C, int ldc, float* T, int ldt, void* workspace,
                            unsigned long long workspace_bytes, void* stream) {
  const int status = check(type, M, N, K, R, S);
  if (status != GEMM_OK) return status;
  if (fused::bad_act(act)) return GEMM_ERR_BAD_ARG;
  if (M == 0 || (N == 0 && T == nullptr)) return GEMM_OK;
  if (bad_ld(ldx, K) || (N > 0 && (bad_ld(ldw, K) || bad_ld(ldc, N))) ||
      (N > 0 && residual && bad_ld(ldr, N)) || (T && bad_ld(ldt, R)) ||
      (S > 0 && (bad_ld(lda, K) || bad_stride(stride_a, S))) ||
      (S > 0 && N > 0 && (bad_ld(ldb, R) || bad_stride(stride_b, S))))
    return GEMM_ERR_BAD_LD;
  if (ids == nullptr || (K > 0 && (X == nullptr || (S > 0 && A == nullptr))) ||
      (N > 0 && (C == nullptr || (K > 0 && W == nullptr) || (S > 0 && B == nullptr))))
    return GEMM_ERR_NULL_POINTER;
  const Mat x0{in16(X), ldx}, w0{in16(W), ldw};
  const Plan p = make_plan(M, N, K, R, S, x0, w0, ldb);
  if (!workspace_ok(p.total(), workspace, workspace_bytes)) return GEMM_ERR_WORKSPACE;
  const int cus = check_device();
  if (cus < 0) return cus;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int fmt = type == GEMM_TYPE_BF16 ? kFmtBF16 : kFmtF16;
  char* ws = static_cast<char*>(workspace);
  half_t* t2 = reinterpret_cast<half_t*>(ws);
  float* factor = reinterpret_cast<float*>(ws + p.t2);
  ws += p.t2 + p.factor;
  const ShrinkArgs sh{in16(X), in16(A), ldx, lda, stride_a, ids, scales, t2, factor, rank_ld2(R),
                      T, ldt, M, K, R, S};
  hipError_t e = launch_shrink(fmt, sh, s);
  if (e != hipSuccess || N == 0) return to_status(e);
  Args16 a{x0.p, w0.p, out16(C), ldx, ldw, ldc, M, N, K};
  a.bias = in16(bias);
  a.res = in16(residual);
  a.ldr = ldr;
  a.act = act;
  a.fmt = fmt;
  LoraExtra y{t2, rank_ld2(R), factor, in16(B), ldb, stride_b, ids, R, S,
                    rank_blocks(R), M, N};
  if (by_rows(M, N, x0, w0)) return to_status(launch_lora_rows(a, y, RowSums(), cus, s));
  PadJobs jobs;
  const Mat x = jobs.add(x0, M, K, ws), w = jobs.add(w0, N, K, ws);
  e = launch_pad(jobs, s);
  if (e != hipSuccess) return to_status(e);
  if (p.b) {
    y.B = reinterpret_cast<half_t*>(ws);
    y.ldb = y.R = 16 * rank_blocks(R);
    y.stride_b = N * y.ldb;
    e = launch_widen(WidenArgs{in16(B), reinterpret_cast<half_t*>(ws), ldb, stride_b, N, R, y.R, S},
                     s);
    if (e != hipSuccess) return to_status(e);
  }
  a.A = x.p;
  a.lda = x.ld;
  a.B = w.p;
  a.ldb = w.ld;
  a.M = pad_rows(M);
  a.N = pad_rows(N);
  a.K = pad_k(K);
  return to_status(launch_lora_tiles(a, y, false, cus, s));
}

MI355TUNE_API unsigned long long gemm_lora_bwd_workspace(int type, int M, int N, int K, int R,
                                                         int S, const void* dC, int lddc,
                                                         const void* W, int ldw, int want_dx,
                                                         int want_da, int want_db) {
  if (check(type, M, N, K, R, S) != GEMM_OK || bad_ld(lddc, N) ||
      (want_dx && M > 0 && K > 0 && bad_ld(ldw, K)) ||
      (((want_da && K > 0) || (want_db && N > 0)) && !can_list(M, S)))
    return 0;
  return plan_bwd(M, N, K, R, S, Mat{in16(dC), lddc}, Mat{in16(W), ldw}, want_dx, want_da, want_db)
      .total();
}

MI355TUNE_API int gemm_lora_bwd(int type, int M, int N, int K, int R, int S, const void* X, int ldx,
                                const void* W, int ldw, const void* A, int lda, long long stride_a,
                                const void* B, int ldb, long long stride_b, const long long* ids,
                                const float* scales, const float* T, int ldt, const void* dC,
                                int lddc, void* dX, int lddx, void* dA, int ldda,
                                long long stride_da, void* dB, int lddb, long long stride_db,
                                void* workspace, unsigned long long workspace_bytes,
                                void* stream) {
  const int status = check(type, M, N, K, R, S);
  if (status != GEMM_OK) return status;
  const Mat c0{in16(dC), lddc}, w0{in16(W), ldw};
  const BwdPlan p = plan_bwd(M, N, K, R, S, c0, w0, dX != nullptr, dA != nullptr, dB != nullptr);
  if (!p.dx && !p.da && !p.db) return GEMM_OK;
  if ((p.da || p.db) && !can_list(M, S)) return GEMM_ERR_BAD_ARG;
  const bool dt = S > 0 && (p.dx || p.da);   // B is read
  if (bad_ld(lddc, N) || (p.dx && (bad_ld(ldw, K) || bad_ld(lddx, K))) ||
      (p.da && (bad_ld(ldx, K) || bad_ld(ldda, K) || bad_out_stride(stride_da, S, R, ldda, K))) ||
      (p.db && (bad_ld(ldt, R) || bad_ld(lddb, R) || bad_out_stride(stride_db, S, N, lddb, R))) ||
      (p.dx && S > 0 && (bad_ld(lda, K) || bad_stride(stride_a, S))) ||
      (dt && (bad_ld(ldb, R) || bad_stride(stride_b, S))))
    return GEMM_ERR_BAD_LD;
  if (M > 0 && (ids == nullptr || (N > 0 && dC == nullptr) ||
                (p.dx && ((N > 0 && W == nullptr) || (S > 0 && A == nullptr))) ||
                (dt && N > 0 && B == nullptr) || (p.da && X == nullptr) ||
                (p.db && T == nullptr)))
    return GEMM_ERR_NULL_POINTER;
  if (!workspace_ok(p.total(), workspace, workspace_bytes)) return GEMM_ERR_WORKSPACE;
  const int cus = check_device();
  if (cus < 0) return cus;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int fmt = type == GEMM_TYPE_BF16 ? kFmtBF16 : kFmtF16;
  char* ws = static_cast<char*>(workspace);
  auto take = [&](size_t bytes) {
    char* at = bytes ? ws : nullptr;
    ws += bytes;
    return at;
  };
  half_t* t2 = reinterpret_cast<half_t*>(take(p.t2));
  float* factor = reinterpret_cast<float*>(take(p.factor));
  float* dt32 = reinterpret_cast<float*>(take(p.dt));
  half_t* at = reinterpret_cast<half_t*>(take(p.at));
  half_t* bt = reinterpret_cast<half_t*>(take(p.bt));
  GroupArgs group{ids, M, S, reinterpret_cast<int*>(take(p.first)),
                  reinterpret_cast<int*>(take(p.rows)), reinterpret_cast<int*>(take(p.steps)),
                  p.grad.steps};
  half_t* pack[2];
  float *step_factor[2], *partial[2];
  for (int i = 0; i < 2; ++i) {
    pack[i] = reinterpret_cast<half_t*>(take(p.pack));
    step_factor[i] = reinterpret_cast<float*>(take(p.step_factor));
    partial[i] = reinterpret_cast<float*>(take(p.partial[i]));
  }
  hipError_t e = hipSuccess;
  const int64_t ldbt = line_ld(round_up(N, 8));
  // B^T as the second operand of dt = dC B, A^T of dX's part, and the lists
  TurnArgs turns[2];
  int count = 0;
  if (M > 0 && dt && N > 0)
    turns[count++] = TurnArgs{in16(B), bt, ldb, stride_b, ldbt, (int64_t)R * ldbt,
                              N, (int)round_up(N, 8), R, S};
  if (p.dx && S > 0)
    turns[count++] = TurnArgs{in16(A), at, lda, stride_a, 16 * rank_blocks(R),
                              (int64_t)K * 16 * rank_blocks(R), R, 16 * rank_blocks(R), K, S};
  const bool listed = p.da || p.db;
  if (listed || count) e = launch_lists(listed ? &group : nullptr, turns, count, s);
  if (e != hipSuccess) return to_status(e);
  if (M > 0 && dt) {
    const ShrinkArgs sh{c0.p, bt, lddc, ldbt, (int64_t)R * ldbt, ids, scales, t2, factor,
                        rank_ld2(R), dt32, R, M, N, R, S};
    e = launch_shrink(fmt, sh, s);
    if (e != hipSuccess) return to_status(e);
  }
  if (p.da || p.db) {
    GradArgs ga;
    ga.g = group;
    ga.scales = scales;
    ga.R = R;
    ga.padded = p.grad.padded;
    ga.groups = p.grad.groups;
    ga.chunks = p.grad.chunks;
    ga.chunk_steps = p.grad.chunk_steps;
    ga.by_adapter = p.grad.by_adapter;
    if (p.da) {
      ga.job[0] = GradJob{dt32, R, in16(X), ldx, K, out16(dA), ldda, stride_da, 0, pack[0],
                          step_factor[0], partial[0], (K + 127) / 128};
    }
    if (p.db) {
      ga.job[1] = GradJob{T, ldt, c0.p, lddc, N, out16(dB), lddb, stride_db, 1, pack[1],
                          step_factor[1], partial[1], (N + 127) / 128};
    }
    e = launch_adapter_grads(fmt, ga, p.grad, s);
    if (e != hipSuccess) return to_status(e);
  }
  LoraExtra y{t2, rank_ld2(R), factor, at, 16 * rank_blocks(R), (int64_t)K * 16 * rank_blocks(R),
              ids, 16 * rank_blocks(R), S, rank_blocks(R), M, K};
  if (p.dx && p.few) {
    float* sum = reinterpret_cast<float*>(ws);
    e = launch_dx(fmt, c0.p, lddc, w0.p, ldw, M, N, K, p.sums, sum, s);
    if (e != hipSuccess) return to_status(e);
    Args16 a{c0.p, w0.p, out16(dX), lddc, ldw, lddx, M, K, 0};
    a.fmt = fmt;
    e = launch_lora_rows(a, y, RowSums{sum, p.sums.ld, p.sums.splits}, cus, s);
  } else if (p.dx) {
    PadJobs jobs;
    Mat c = c0, w = w0;
    if (p.copy_c) c = jobs.copy(c0, M, N, ws);
    if (p.copy_w) {
      // as many rows as dC's copy has columns
      w = jobs.copy(w0, N, K, ws);
      const int i = jobs.count - 1;
      jobs.job[i].rows_p = pad_k(pad_rows(N));
      const int64_t pieces = (int64_t)jobs.job[i].rows_p * (jobs.job[i].cols_p / 8);
      jobs.blocks[i] = (i ? jobs.blocks[i - 1] : 0) + (pieces + 255) / 256;
    }
    e = launch_pad(jobs, s);
    if (e != hipSuccess) return to_status(e);
    Args16 a{c.p, w.p, out16(dX), c.ld, w.ld, lddx, pad_rows(M), pad_k(K), pad_k(N)};
    a.fmt = fmt;
    if (p.tail) {
      y.tail = reinterpret_cast<half_t*>(ws);
      e = launch_tail(TailArgs{c0.p, reinterpret_cast<half_t*>(ws), lddc, M, a.M, a.K}, s);
      if (e != hipSuccess) return to_status(e);
    }
    e = launch_lora_tiles(a, y, true, cus, s);
  }
  return to_status(e);
}

}  // extern "C"

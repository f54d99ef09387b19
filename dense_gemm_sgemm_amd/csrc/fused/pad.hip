// Padded copies of 16-bit matrices, for operands that the tile kernels cannot
// read in place (rows not at 16-byte addresses, fewer rows or columns than a
// tile).  One thread a 16-byte piece of the copy; bound by HBM: the source is
// read and the copy written once.
#include "fused.hpp"

namespace mi355gemm {
namespace fused {
namespace {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
constexpr int kThreads = 256;

__global__ __launch_bounds__(kThreads) void pad_kernel(PadJobs jobs, int64_t base) {
  int64_t block = base + blockIdx.x;
  int which = 0;
  while (which + 1 < jobs.count && block >= jobs.blocks[which]) ++which;
  if (which > 0) block -= jobs.blocks[which - 1];
  const PadJob& j = jobs.job[which];
  const int chunks = j.cols_p / 8;
  const int64_t t = block * kThreads + threadIdx.x;
  if (t >= (int64_t)j.rows_p * chunks) return;
  const int64_t r = t / chunks;
  const int c = (int)(t % chunks) * 8;
  h8 v = {};
  if (r < j.rows) {
    const half_t* s = j.src + r * j.lds + c;
    if (c + 8 <= j.cols) {
      __builtin_memcpy(&v, s, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e < j.cols) v[e] = s[e];
    }
  }
  *(h8*)(j.dst + r * j.ldd + c) = v;
}

}  // namespace

Mat PadJobs::add(Mat m, int rows, int K, char*& dst) {
  return needs_copy(m.p, m.ld, rows, K) ? copy(m, rows, K, dst) : m;
}

Mat PadJobs::copy(Mat m, int rows, int K, char*& dst) {
  PadJob& j = job[count];
  j.src = m.p;
  j.dst = reinterpret_cast<half_t*>(dst);
  j.lds = m.ld;
  j.ldd = line_ld(pad_k(K));
  j.rows = rows;
  j.cols = K;
  j.rows_p = pad_rows(rows);
  j.cols_p = pad_k(K);
  const int64_t pieces = (int64_t)j.rows_p * (j.cols_p / 8);
  blocks[count] = (count ? blocks[count - 1] : 0) + (pieces + kThreads - 1) / kThreads;
  ++count;
  dst += copy_bytes(rows, K);
  return Mat{j.dst, j.ldd};
}

hipError_t launch_pad(const PadJobs& jobs, hipStream_t stream) {
  if (jobs.count == 0) return hipSuccess;
  return launch_tiles((const void*)pad_kernel, jobs, jobs.blocks[jobs.count - 1], kThreads, 0,
                      stream);
}

}  // namespace fused
}  // namespace mi355gemm

// The last step of a product whose K was cut into ranges or pieces: the
// ranges' fp32 sums added in order, scaled and rounded.  Bound by HBM (the
// sums are read once).
#include "fused.hpp"

namespace mi355gemm {
namespace fused {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
constexpr int kThreads = 256;

struct SumArgs {
  const float* sum;
  half_t* out;
  const float* scale;
  int64_t ld_sum, split_stride, ldo;
  int splits, M, N;
};

// One thread 4 columns of a row (the sums' rows are padded to whole quads).
template <int FMT>
__global__ __launch_bounds__(kThreads) void sum_kernel(SumArgs p, int64_t base) {
  const int quads = (p.N + 3) / 4;
  const int64_t t = (base + blockIdx.x) * kThreads + threadIdx.x;
  if (t >= (int64_t)p.M * quads) return;
  const int64_t m = t / quads;
  const int n = (int)(t % quads) * 4;
  const float* src = p.sum + m * p.ld_sum + n;
  f4 s = *(const f4*)src;
  int k = 1;
  for (; k + 4 <= p.splits; k += 4) {   // four loads in flight
    f4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = *(const f4*)(src + (k + u) * p.split_stride);
#pragma unroll
    for (int u = 0; u < 4; ++u) s += v[u];
  }
  for (; k < p.splits; ++k) s += *(const f4*)(src + k * p.split_stride);
  if (p.scale) s *= p.scale[1];
  h4 o;
#pragma unroll
  for (int v = 0; v < 4; ++v) o[v] = f32_to_word<FMT>(s[v]);
  half_t* dst = p.out + m * p.ldo + n;
  if (n + 4 <= p.N) {
    __builtin_memcpy(dst, &o, 8);
  } else {
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (n + v < p.N) dst[v] = o[v];
  }
}

}  // namespace

hipError_t launch_sums(int fmt, const FusedExtra& x, int splits, half_t* out, int64_t ldo, int M,
                       int N, hipStream_t stream) {
  const SumArgs p{x.sum, out, x.scale, x.ld_sum, x.split_stride, ldo, splits, M, N};
  const int64_t threads = (int64_t)M * ((N + 3) / 4);
  return launch_tiles(fmt == kFmtBF16 ? (const void*)sum_kernel<kFmtBF16>
                                      : (const void*)sum_kernel<kFmtF16>,
                      p, (threads + kThreads - 1) / kThreads, kThreads, 0, stream);
}

}  // namespace fused
}  // namespace mi355gemm

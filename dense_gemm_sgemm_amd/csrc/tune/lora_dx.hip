// dC W for few rows, W [N][K] summed over its rows: bound by streaming W once for
// 64 rows.  W's rows are the summed index, so a lane loads 8 rows x 8 columns in
// 16-byte pieces and exchanges them in registers (turn8), as for the adapters'
// gradients; dC's rows are fragments as they lie.  No LDS but for adding up the
// waves, no copies, any alignment.  bf16, N and K of 4096: 16 us for 64 rows, 23 for
// 256 (the weights in cache).
//
// A workgroup takes 64 rows (at most), 128 columns and a range of N, which its
// waves share in steps of 32; it leaves fp32 sums, [range][row][column], that the
// kernel with the adapters' part (lora_rows.hip) adds up.
#include "fused/skinny.hpp"
#include "tune.hpp"

namespace mi355gemm {
namespace tune {
namespace {

using namespace fused::skinny;
constexpr int kThreads = 256, kWaves = 4, kCols = 128;

struct DxArgs {
  const half_t *dC, *W;
  int64_t lddc, ldw, ld_sum;
  int M, N, K, blocks, splits, per;   // per: steps of 32 of N in a range
  float* sum;
};

template <int FMT, int MT>
__global__ __launch_bounds__(kThreads, MT == 4 ? 2 : 1) void dx_kernel(DxArgs p, int64_t base) {
  __shared__ f4 lds[(kWaves - 1) * 8 * 64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, j = lane & 15;
  int64_t id = base + blockIdx.x;
  const int block = (int)(id % p.blocks);
  id /= p.blocks;
  const int range = (int)(id % p.splits), m0 = (int)(id / p.splits) * 64;
  const int col = block * kCols + 8 * j;
  const int steps = (p.N + 31) / 32;
  const int s0 = range * p.per, s1 = s0 + p.per < steps ? s0 + p.per : steps;
  const half_t* c[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int m = m0 + 16 * t + j;   // rows past M repeat the last one, unstored
    c[t] = p.dC + (int64_t)(m < p.M ? m : p.M - 1) * p.lddc;
  }
  f4 acc[MT][8];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[t][e] = f4{0.f, 0.f, 0.f, 0.f};
  auto load = [&](int s, h8 (&x)[8], h8 (&d)[MT]) __attribute__((always_inline)) {
    const int n = 32 * s + 8 * g;
    const half_t* w = p.W + (int64_t)n * p.ldw + col;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = h8{};
      if (n + i < p.N && col < p.K) {
        if (col + 8 <= p.K) {
          __builtin_memcpy(&x[i], w + i * p.ldw, 16);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (col + e < p.K) x[i][e] = w[i * p.ldw + e];
        }
      }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) d[t] = load_x<true>(c[t], n, p.N);
  };
  // (64 rows leave no registers for a step ahead, but two waves a SIMD)
  constexpr bool kAhead = MT < 4;
  h8 x[8], nx[8], d[MT], nd[MT];
  int s = s0 + wave;
  if (kAhead && s < s1) load(s, x, d);
  for (; s < s1; s += kWaves) {
    if (!kAhead) load(s, x, d);
    if (kAhead && s + kWaves < s1) load(s + kWaves, nx, nd);
    turn8(x);
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[t][e] = mfma16<FMT>(d[t], x[e], acc[t][e]);
    if (kAhead) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = nx[i];
#pragma unroll
      for (int t = 0; t < MT; ++t) d[t] = nd[t];
    }
  }
  add_up<MT>(acc, lds, wave, lane);
  if (wave > 0 || col >= p.K) return;
  // acc[t][e][v]: row 16 t + 4 g + v, column col + e (rows of the sums are padded to
  // eights)
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int m = m0 + 16 * t + 4 * g + v;
      if (m >= p.M) continue;
      float* out = p.sum + ((int64_t)range * p.M + m) * p.ld_sum + col;
      f4 a, b;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = acc[t][e][v];
        b[e] = acc[t][4 + e][v];
      }
      *(f4*)out = a;
      *(f4*)(out + 4) = b;
    }
}

template <int FMT>
const void* pick(int M) {
  return M <= 16   ? (const void*)dx_kernel<FMT, 1>
         : M <= 32 ? (const void*)dx_kernel<FMT, 2>
                   : (const void*)dx_kernel<FMT, 4>;
}

}  // namespace

// Ranges for some 512 workgroups, of at least two turns of the waves each; fewer
// where their sums are many.
DxPlan plan_dx(int M, int N, int K) {
  const int64_t blocks = ((int64_t)K + kCols - 1) / kCols * (((int64_t)M + 63) / 64);
  const int steps = (N + 31) / 32;
  DxPlan p;
  p.splits = (int)std::max<int64_t>(
      1, std::min<int64_t>(
             {M > 32 ? 8 : 16, 512 / std::max<int64_t>(1, blocks), steps / (2 * kWaves)}));
  p.per = (steps + p.splits - 1) / p.splits;
  p.splits = p.per ? (steps + p.per - 1) / p.per : 1;
  p.ld = round_up(K, 8);
  p.bytes = round256((size_t)p.splits * M * p.ld * sizeof(float));
  return p;
}

hipError_t launch_dx(int fmt, const half_t* dC, int64_t lddc, const half_t* W, int64_t ldw, int M,
                     int N, int K, const DxPlan& plan, float* sum, hipStream_t stream) {
  const int blocks = (K + kCols - 1) / kCols;
  const DxArgs p{dC, W, lddc, ldw, plan.ld, M, N, K, blocks, plan.splits, plan.per, sum};
  return launch_tiles(fmt == kFmtBF16 ? pick<kFmtBF16>(M) : pick<kFmtF16>(M), p,
                      (int64_t)blocks * plan.splits * ((M + 63) / 64), kThreads, 0, stream);
}

}  // namespace tune
}  // namespace mi355gemm

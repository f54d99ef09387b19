// The gated product for few rows of X (decode steps): both weights streamed
// from HBM once, bound by that.  A wave loads 16 rows x 128 k of Wg and of Wu
// (16 bytes a lane and step of 32 k) one chunk ahead of the products; see
// skinny.hpp for the layout.
#include "skinny.hpp"

namespace mi355gemm {
namespace fused {
namespace {

using namespace skinny;

constexpr int kSteps = 4;              // steps of 32 k in a chunk
constexpr int kChunk = 32 * kSteps;
constexpr int kMaxWaves = 8;

struct RowsArgs {
  const half_t *X, *Wg, *Wu;
  half_t *H, *G, *U;
  int64_t ldx, ldwg, ldwu, ldh, ldg, ldu;
  int M, N, K, act, waves;
};

template <bool TAIL>
__device__ __forceinline__ void load_chunk(const half_t* g, const half_t* u, int k, int K,
                                           h8 (&w)[2][kSteps]) {
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    w[0][s] = load_x<TAIL>(g, k + 32 * s, K);
    w[1][s] = load_x<TAIL>(u, k + 32 * s, K);
  }
}

template <int FMT, int MT, bool TAIL>
__device__ __forceinline__ void multiply(const half_t* const (&xrow)[MT], int k, int K,
                                         const h8 (&w)[2][kSteps], f4 (&acc)[2 * MT]) {
  h8 x[MT][kSteps];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int s = 0; s < kSteps; ++s) x[t][s] = load_x<TAIL>(xrow[t], k + 32 * s, K);
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      acc[t] = mfma16<FMT>(x[t][s], w[0][s], acc[t]);
      acc[MT + t] = mfma16<FMT>(x[t][s], w[1][s], acc[MT + t]);
    }
}

template <int FMT, int MT>
__global__ __launch_bounds__(64 * kMaxWaves) void gated_rows_kernel(RowsArgs p, int64_t base) {
  extern __shared__ __attribute__((aligned(16))) float lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, quarter = lane >> 4;
  const int n = (int)(base + blockIdx.x) * 16 + r;
  const int row = n < p.N ? n : p.N - 1;   // rows past N repeat the last one, unstored
  const half_t* wg = p.Wg + row * p.ldwg + 8 * quarter;
  const half_t* wu = p.Wu + row * p.ldwu + 8 * quarter;
  const half_t* xrow[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int m = 16 * t + r;
    xrow[t] = p.X + (m < p.M ? m : p.M - 1) * p.ldx + 8 * quarter;   // as for W
  }
  f4 acc[2 * MT];
#pragma unroll
  for (int t = 0; t < 2 * MT; ++t) acc[t] = f4{0.f, 0.f, 0.f, 0.f};

  // (pointers and K both moved on by the lane's 8 quarter)
  const int K = p.K - 8 * quarter, chunks = p.K / kChunk;
  h8 cur[2][kSteps], nxt[2][kSteps];
  int c = wave;
  if (c < chunks) load_chunk<false>(wg, wu, c * kChunk, K, cur);
  for (; c < chunks; c += p.waves) {
    if (c + p.waves < chunks) load_chunk<false>(wg, wu, (c + p.waves) * kChunk, K, nxt);
    multiply<FMT, MT, false>(xrow, c * kChunk, K, cur, acc);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      cur[0][s] = nxt[0][s];
      cur[1][s] = nxt[1][s];
    }
  }
  if (chunks * kChunk < p.K && wave == chunks % p.waves) {
    load_chunk<true>(wg, wu, chunks * kChunk, K, cur);
    multiply<FMT, MT, true>(xrow, chunks * kChunk, K, cur, acc);
  }

  add_waves<2 * MT>(acc, lds, wave, lane, p.waves);
  if (wave > 0 || n >= p.N) return;
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t m = 16 * t + 4 * quarter + v;
      if (m >= p.M) continue;
      const float g = acc[t][v], u = acc[MT + t][v];
      p.H[m * p.ldh + n] = f32_to_word<FMT>(epi_act(g, p.act) * u);
      if (p.G) p.G[m * p.ldg + n] = f32_to_word<FMT>(g);
      if (p.U) p.U[m * p.ldu + n] = f32_to_word<FMT>(u);
    }
}

template <int FMT>
const void* pick(int M) {
  return M <= 16   ? (const void*)gated_rows_kernel<FMT, 1>
         : M <= 32 ? (const void*)gated_rows_kernel<FMT, 2>
                   : (const void*)gated_rows_kernel<FMT, 4>;
}

}  // namespace

hipError_t launch_gated_rows(const Args16& a, const FusedExtra& x, int cus, hipStream_t stream) {
  RowsArgs p{a.A,   a.B,    x.B2,  a.C,   x.C2,  x.C3, a.lda, a.ldb, x.ldb2,
             a.ldc, x.ldc2, x.ldc3, a.M, a.N, a.K, a.act, 1};
  const int mt = a.M <= 16 ? 1 : a.M <= 32 ? 2 : 4;
  const int64_t wgs = ((int64_t)a.N + 15) / 16;
  const int chunks = std::max(1, (int)(((int64_t)a.K + kChunk - 1) / kChunk));
  p.waves = waves_for(wgs, chunks, kMaxWaves, cus);
  return launch_tiles(a.fmt == kFmtBF16 ? pick<kFmtBF16>(a.M) : pick<kFmtF16>(a.M), p, wgs,
                      64 * p.waves, (unsigned)((p.waves - 1) * 2 * mt * 64 * sizeof(f4)), stream);
}

}  // namespace fused
}  // namespace mi355gemm

// The gated product for few rows of X (decode steps): both weights streamed
// from HBM once for 64 rows, bound by that.  A wave loads 16 rows x 128 or 64 k of Wg and of Wu
// (16 bytes a lane and step of 32 k) one chunk ahead of the products; see
// skinny.hpp for the layout.
#include "skinny.hpp"

namespace mi355gemm {
namespace fused {
namespace {

using namespace skinny;

// Steps of 32 k in a chunk: four where the weights are all there is to load,
// two where X and its sums need the registers (one token, 16384 x 4096: 45.8
// against 47.9 us; 24 rows, 8192 x 2048: 17.7 against 14.2).
constexpr int steps_of(int mt) { return mt == 1 ? 4 : 2; }
constexpr int kMaxWaves = 8;

struct RowsArgs {
  const half_t *X, *Wg, *Wu;
  half_t *H, *G, *U;
  int64_t ldx, ldwg, ldwu, ldh, ldg, ldu;
  int M, N, K, act, waves;
};

template <bool TAIL, int kSteps>
__device__ __forceinline__ void load_chunk(const half_t* g, const half_t* u, int k, int K,
                                           h8 (&w)[2][kSteps]) {
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    w[0][s] = load_x<TAIL>(g, k + 32 * s, K);
    w[1][s] = load_x<TAIL>(u, k + 32 * s, K);
  }
}

template <int FMT, int MT, int kSteps>
__device__ __forceinline__ void multiply(const h8 (&x)[MT][kSteps], const h8 (&w)[2][kSteps],
                                         f4 (&acc)[2 * MT]) {
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
  constexpr int kSteps = steps_of(MT), kChunk = 32 * kSteps;
  typedef XStage<MT, kChunk> Stage;
  __shared__ __attribute__((aligned(16))) unsigned char
      lds[kMaxWaves * (Stage::kBytes > 2 * MT * 1024 ? Stage::kBytes : 2 * MT * 1024)];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, quarter = lane >> 4;
  const int64_t id = base + blockIdx.x, groups_n = (p.N + 15) / 16;
  const int m0 = (int)(id / groups_n) * 64;
  const int n = (int)(id % groups_n) * 16 + r;
  const int row = n < p.N ? n : p.N - 1;   // rows past N repeat the last one, unstored
  const half_t* wg = p.Wg + row * p.ldwg + 8 * quarter;
  const half_t* wu = p.Wu + row * p.ldwu + 8 * quarter;
  f4 acc[2 * MT];
#pragma unroll
  for (int t = 0; t < 2 * MT; ++t) acc[t] = f4{0.f, 0.f, 0.f, 0.f};

  // (pointers and K both moved on by the lane's 8 quarter)
  const int K = p.K - 8 * quarter, chunks = p.K / kChunk;
  h8 cur[2][kSteps], nxt[2][kSteps], x[MT][kSteps];
  Stage stage;
  unsigned char* buf = lds + wave * Stage::kBytes;
  auto read_x = [&]() __attribute__((always_inline)) {
    stage.store(buf, lane, [](h8 v) { return v; });
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int s = 0; s < kSteps; ++s) x[t][s] = Stage::read(buf, t, r, 32 * s + 8 * quarter);
  };
  int c = wave;
  if (c < chunks) {
    stage.template load<false>(p.X, p.ldx, m0, p.M, c * kChunk, p.K, lane);
    load_chunk<false, kSteps>(wg, wu, c * kChunk, K, cur);
  }
  for (; c < chunks; c += p.waves) {
    read_x();
    if (c + p.waves < chunks) {
      stage.template load<false>(p.X, p.ldx, m0, p.M, (c + p.waves) * kChunk, p.K, lane);
      load_chunk<false, kSteps>(wg, wu, (c + p.waves) * kChunk, K, nxt);
    }
    multiply<FMT, MT, kSteps>(x, cur, acc);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      cur[0][s] = nxt[0][s];
      cur[1][s] = nxt[1][s];
    }
  }
  if (chunks * kChunk < p.K && wave == chunks % p.waves) {
    stage.template load<true>(p.X, p.ldx, m0, p.M, chunks * kChunk, p.K, lane);
    load_chunk<true, kSteps>(wg, wu, chunks * kChunk, K, cur);
    read_x();
    multiply<FMT, MT, kSteps>(x, cur, acc);
  }

  // (the sums take the place of X)
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  add_waves<2 * MT>(acc, reinterpret_cast<float*>(lds), wave, lane, p.waves);
  if (wave > 0 || n >= p.N) return;
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t m = m0 + 16 * t + 4 * quarter + v;
      if (m >= p.M) continue;
      const float g = acc[t][v], u = acc[MT + t][v];
      p.H[m * p.ldh + n] = f32_to_word<FMT>(gate_act(g, p.act) * u);
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
  const int64_t wgs = ((int64_t)a.N + 15) / 16 * (((int64_t)a.M + 63) / 64);
  const int chunk = 32 * steps_of(a.M <= 16 ? 1 : 2);
  const int chunks = std::max(1, (int)(((int64_t)a.K + chunk - 1) / chunk));
  p.waves = waves_for(wgs, chunks, kMaxWaves, cus);
  return launch_tiles(a.fmt == kFmtBF16 ? pick<kFmtBF16>(a.M) : pick<kFmtF16>(a.M), p, wgs,
                      64 * p.waves, 0, stream);
}

}  // namespace fused
}  // namespace mi355gemm

// A product with adapters for few rows of X (decode steps): W streamed from HBM
// once for 64 rows, bound by that (skinny.hpp has the layout; here W goes through a
// wave's own copy in LDS too, so that its loads cover whole lines: fp16, N and K of
// 4096, 1 row 8.8 -> 7.2 us, 4.7 TB/s; 32 rows 11.5 -> 10.5; 64 x 8192 x 8192 47 ->
// 42; 19 odd rows of 5669, N 2545: 29 -> 19).  64 values of K a turn for more than 16
// rows, so that LDS holds two workgroups (N 14336, 32 rows: 36 -> 29 us).  The adapters'
// second product comes before the waves' sums are added: each wave takes every
// so many of the adapters that the rows name, multiplies t (tune.hpp) with 16 of
// the adapter's rows of B and keeps the sums of the rows that are its own, apart
// from the projection's: one wave has them, so that a row's result does not
// depend on the rows beside it.
#include "fused/skinny.hpp"
#include "tune.hpp"

namespace mi355gemm {
namespace tune {
namespace {

using namespace fused::skinny;

constexpr int kSteps = 4, kChunk = 32 * kSteps, kMaxWaves = 8;

struct RowsArgs {
  Args16 p;
  LoraExtra x;
  RowSums sums;
  int waves;
};

// Columns at .. at + 7 of a row of R, zeros past it.  `room`: elements from the
// row's start to the end of its matrix, up to which a whole 16-byte piece may
// be loaded; what lies past the row is masked.
__device__ __forceinline__ h8 load_ranks(const half_t* row, int at, int R, int64_t room) {
  h8 v = {};
  if (at + 8 <= room) {
    __builtin_memcpy(&v, row + at, 16);
    if (at + 8 > R) {
      typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
      u32x4 w = __builtin_bit_cast(u32x4, v);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = at + 2 * e + 1 < R ? w[e] : at + 2 * e < R ? w[e] & 0xFFFFu : 0u;
      v = __builtin_bit_cast(h8, w);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (at + e < R) v[e] = row[at + e];
  }
  return v;
}

template <int FMT, int MT>
__global__ __launch_bounds__(64 * kMaxWaves) void lora_rows_kernel(RowsArgs args, int64_t base) {
  constexpr int kS = MT == 1 ? kSteps : 2, kC = 32 * kS;
  typedef XStage<MT, kC> Stage;
  typedef XStage<1, kC> WStage;
  constexpr int kBytes = Stage::kBytes + WStage::kBytes;
  __shared__ __attribute__((aligned(16))) unsigned char
      lds[kMaxWaves * (kBytes > 2 * MT * 1024 ? kBytes : 2 * MT * 1024)];
  const Args16& p = args.p;
  const LoraExtra& y = args.x;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, quarter = lane >> 4;
  const int64_t id = base + blockIdx.x, groups_n = (p.N + 15) / 16;
  const int m0 = (int)(id / groups_n) * 64;
  const int n = (int)(id % groups_n) * 16 + r;
  const int row = n < p.N ? n : p.N - 1;   // rows past N repeat the last one, unstored
  f4 acc[2 * MT];   // the projection's, then the adapters'
#pragma unroll
  for (int t = 0; t < 2 * MT; ++t) acc[t] = f4{0.f, 0.f, 0.f, 0.f};

  const int chunks = p.K / kC;
  Stage stage;
  WStage wstage;
  unsigned char* buf = lds + wave * kBytes;
  const int n0 = (int)(id % groups_n) * 16;
  auto load = [&](int k, auto tail) __attribute__((always_inline)) {
    constexpr bool kTail = decltype(tail)::value;
    wstage.template load<kTail>(p.B, p.ldb, n0, p.N, k, p.K, lane);
    stage.template load<kTail>(p.A, p.lda, m0, p.M, k, p.K, lane);
  };
  auto store = [&]() __attribute__((always_inline)) {
    auto as_is = [](h8 v) { return v; };
    stage.store(buf, lane, as_is);
    wstage.store(buf + Stage::kBytes, lane, as_is);
  };
  auto multiply = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < kS; ++s) {
      const h8 wv = WStage::read(buf + Stage::kBytes, 0, r, 32 * s + 8 * quarter);
#pragma unroll
      for (int t = 0; t < MT; ++t)
        acc[t] = mfma16<FMT>(Stage::read(buf, t, r, 32 * s + 8 * quarter), wv, acc[t]);
    }
    asm volatile("" ::: "memory");
  };
  if (args.sums.sum) {
    // (the waves share the ranges; rows past M repeat the last one, unstored)
    for (int s = wave; s < args.sums.ranges; s += args.waves)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int m = m0 + 16 * t + 4 * quarter + v;
          acc[t][v] +=
              args.sums.sum[((int64_t)s * p.M + (m < p.M ? m : p.M - 1)) * args.sums.ld_sum + row];
        }
  }
  // The adapters: lane l stands for row m0 + l.  What the first block of ranks and
  // the wave's first adapters need is loaded before the products.
  const int mine = m0 + lane < p.M ? adapter_of(y.ids, m0 + lane, y.S) : -1;
  const uint64_t named = __ballot(mine >= 0);
  uint64_t pending = named;
  int turn = 0, block = 0;
  constexpr int kAhead = 4;
  h8 tv[MT], bv[kAhead];
  float factor[MT][4];
  uint64_t rows[kAhead] = {};
  auto load_t = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      // (rows without an adapter, and past M: any values, dropped below)
      const int m = m0 + 16 * t + r;
      tv[t] = *(const h8*)(y.t2 + (m < p.M ? m : p.M - 1) * y.ld2 + 32 * block + 8 * quarter);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t i = m0 + 16 * t + 4 * quarter + v;
        factor[t][v] = y.factor[(i < p.M ? i : p.M - 1) * y.blocks + block];
      }
    }
  };
  // the wave's next adapters: every so many of those that the rows name
  auto load_b = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      rows[q] = 0;
      bv[q] = h8{};
      int a = 0;
      while (pending && !rows[q]) {
        a = __builtin_amdgcn_readlane(mine, __builtin_ctzll(pending));
        const uint64_t own = __ballot(mine == a);
        pending &= ~own;
        if (turn == wave) rows[q] = own;
        turn = turn + 1 == args.waves ? 0 : turn + 1;
      }
      if (rows[q])
        bv[q] = load_ranks(y.B + a * y.stride_b + (int64_t)row * y.ldb,
                           16 * block + 8 * (quarter & 1), y.R,
                           (int64_t)(p.N - 1 - row) * y.ldb + y.R);
    }
  };
  if (named) {
    load_t();
    load_b();
  }
  int c = wave;
  if (c < chunks) load(c * kC, std::false_type());
  for (; c < chunks; c += args.waves) {
    store();
    if (c + args.waves < chunks) load((c + args.waves) * kC, std::false_type());
    multiply();
  }
  if (chunks * kC < p.K && wave == chunks % args.waves) {
    load(chunks * kC, std::true_type());
    store();
    multiply();
  }

  while (named) {
#pragma unroll
    for (int q = 0; q < kAhead; ++q)
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        if (!(rows[q] >> (16 * t) & 0xFFFF)) continue;
        const f4 s = mfma16<FMT>(tv[t], bv[q], f4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (rows[q] >> (16 * t + 4 * quarter + v) & 1) acc[MT + t][v] += factor[t][v] * s[v];
      }
    if (!pending) {
      if (++block == y.blocks) break;
      pending = named;
      turn = 0;
      load_t();
    }
    load_b();
  }

  // (the sums take the place of X)
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  add_waves<2 * MT>(acc, reinterpret_cast<float*>(lds), wave, lane, args.waves);
  if (wave > 0) return;
  const uint64_t unknown = __ballot(mine == -2);
  if (n >= p.N) return;
  const float bias = p.bias ? word_to_f32<FMT>(p.bias[n]) : 0.f;
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int i = 16 * t + 4 * quarter + v;
      const int64_t m = m0 + i;
      if (m >= p.M) continue;
      float z = unknown >> i & 1 ? __builtin_nanf("") : acc[t][v] + acc[MT + t][v];
      z = gate_act(z + bias, p.act);
      if (p.res) z += word_to_f32<FMT>(p.res[m * p.ldr + n]);
      p.C[m * p.ldc + n] = f32_to_word<FMT>(z);
    }
}

template <int FMT>
const void* pick(int M) {
  return M <= 16   ? (const void*)lora_rows_kernel<FMT, 1>
         : M <= 32 ? (const void*)lora_rows_kernel<FMT, 2>
                   : (const void*)lora_rows_kernel<FMT, 4>;
}

}  // namespace

hipError_t launch_lora_rows(const Args16& a, const LoraExtra& x, const RowSums& sums, int cus,
                            hipStream_t stream) {
  RowsArgs p{a, x, sums, 1};
  if (sums.sum) p.p.K = 0;
  const int64_t wgs = ((int64_t)a.N + 15) / 16 * (((int64_t)a.M + 63) / 64);
  const int chunk = a.M <= 16 ? kChunk : kChunk / 2;
  const int chunks = std::max(1, (int)(((int64_t)a.K + chunk - 1) / chunk));
  p.waves = sums.sum ? std::max(1, std::min(kMaxWaves, sums.ranges))
                     : waves_for(wgs, chunks, kMaxWaves, cus);
  return launch_tiles(a.fmt == kFmtBF16 ? pick<kFmtBF16>(a.M) : pick<kFmtF16>(a.M), p, wgs,
                      64 * p.waves, 0, stream);
}

}  // namespace tune
}  // namespace mi355gemm

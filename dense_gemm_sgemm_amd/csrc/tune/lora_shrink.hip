// t[m][r] = sum_k X[m][k] A_a[r][k] with a the adapter of row m: each adapter's
// ranks are few, so the product streams X once and the adapters that its rows
// name once a block of 16 rows (from L2 where neighbours share them).
//
// A workgroup takes 16 rows, one of the adapters they name and up to 64 ranks;
// its eight waves share K out in turns of 128 (64 for more ranks), the next turn's
// loads in flight, and add up through LDS: with few rows the time is a few memory
// latencies.  Both operands go through a copy in LDS that is each wave's own, so that
// a load covers whole lines: read straight into the fragments' layout, 16 rows x 64
// bytes, the loads themselves were the time (bf16, K 4096, 16 ranks: 64 rows 12.8 ->
// 8.6 us, 4096 rows 20 -> 9.6 us, 3.5 TB/s; 19 odd rows of 5669: 47 -> 18 us), and
// sixteen waves with half of the registers spilled (9.6 -> 20 us).  Rows of other
// adapters are multiplied along and dropped.
// Only the GPU knows the ids, so a block of rows has places for adapters, up to
// 16 while the launch is small: a workgroup takes its place's adapter and every
// so many after it, and ends if there is none (256 blocks of 4096 rows with 16
// places: 10 us for workgroups that end at once).
#include "fused/skinny.hpp"
#include "tune.hpp"

namespace mi355gemm {
namespace tune {
namespace {

using namespace fused::skinny;

constexpr int kWaves = 8, kMaxSlots = 16, kWorkgroups = 512;
constexpr int steps_of(int rb) { return rb == 1 ? 4 : 2; }

// One adapter's ranks first .. of the 16 rows from m0 (`rows`: its own).
template <int FMT, int RB>
__device__ __forceinline__ void shrink_one(const ShrinkArgs& p, unsigned char* lds, int a,
                                           uint32_t rows, int m0, int first, int lane, int wave) {
  constexpr int kSteps = steps_of(RB), kChunk = 32 * kSteps;
  typedef XStage<1, kChunk> Stage;
  const int r = lane & 15, quarter = lane >> 4;
  const half_t* w = p.A + a * p.stride_a;
  f4 acc[RB];
#pragma unroll
  for (int q = 0; q < RB; ++q) acc[q] = f4{0.f, 0.f, 0.f, 0.f};
  const int chunks = p.K / kChunk;
  Stage stage[2][1 + RB];   // X, then the ranks
  unsigned char* buf = lds + wave * (1 + RB) * Stage::kBytes;
  // where the lane's pieces of a turn begin (rows past M and ranks past R repeat the
  // last one and count as zeros)
  constexpr int kLoads = Stage::kLoads;
  const half_t* at[1 + RB][kLoads];
  const int column = lane % Stage::kPieces * 8;
#pragma unroll
  for (int e = 0; e < kLoads; ++e) {
    const int i = e * Stage::kRows + lane / Stage::kPieces, m = m0 + i;
    at[0][e] = p.X + (m < p.M ? m : p.M - 1) * p.ldx + column;
#pragma unroll
    for (int q = 0; q < RB; ++q) {
      const int n = first + 16 * q + i;
      at[1 + q][e] = w + (n < p.R ? n : p.R - 1) * p.lda + column;
    }
  }
  auto load = [&](int set, int k, auto tail) __attribute__((always_inline)) {
    // (k of unknown origin: one address kept a piece, not one a piece and set)
    asm volatile("" : "+s"(k));
#pragma unroll
    for (int q = 0; q < 1 + RB; ++q)
#pragma unroll
      for (int e = 0; e < kLoads; ++e)
        stage[set][q].v[e] = load_x<decltype(tail)::value>(at[q][e], k, p.K - column);
  };
  auto multiply = [&](int set) __attribute__((always_inline)) {
    auto as_is = [](h8 v) { return v; };
#pragma unroll
    for (int q = 0; q < 1 + RB; ++q) stage[set][q].store(buf + q * Stage::kBytes, lane, as_is);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const h8 xv = Stage::read(buf, 0, r, 32 * s + 8 * quarter);
#pragma unroll
      for (int q = 0; q < RB; ++q)
        acc[q] = mfma16<FMT>(
            xv, Stage::read(buf + (1 + q) * Stage::kBytes, 0, r, 32 * s + 8 * quarter), acc[q]);
    }
    asm volatile("" ::: "memory");
  };
  // two turns at a time, so that the sets are named by constants
  int c = wave;
  if (c < chunks) load(0, c * kChunk, std::false_type());
  for (; c < chunks; c += 2 * kWaves) {
    const bool second = c + kWaves < chunks;
    if (second) load(1, (c + kWaves) * kChunk, std::false_type());
    multiply(0);
    if (c + 2 * kWaves < chunks) load(0, (c + 2 * kWaves) * kChunk, std::false_type());
    if (second) multiply(1);
  }
  if (chunks * kChunk < p.K && wave == chunks % kWaves) {
    load(0, chunks * kChunk, std::true_type());
    multiply(0);
  }
  __syncthreads();   // the sums take the place of the operands
  add_waves<RB>(acc, reinterpret_cast<float*>(lds), wave, lane, kWaves);
  if (wave > 0) return;

  const int blocks = rank_blocks(p.R);
  // acc[q][v]: row 4 quarter + v, rank first + 16 q + r
#pragma unroll
  for (int q = 0; q < RB; ++q)
    if (first + 16 * q + r >= p.R) acc[q] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int i = 4 * quarter + v;
    const int64_t m = m0 + i;
    const bool live = rows >> i & 1;
    if (p.t32 && live) {
#pragma unroll
      for (int q = 0; q < RB; ++q)
        if (first + 16 * q + r < p.R) p.t32[m * p.ldt + first + 16 * q + r] = acc[q][v];
    }
    if (!p.t2) continue;
    const float scale = p.scales ? p.scales[a] : 1.f;
#pragma unroll
    for (int q = 0; q < RB; ++q) {
      const float t = acc[q][v];
      float top = fabsf(t), up, down;
      if (!(top < __builtin_inff())) top = 0.f;
#pragma unroll
      for (int k = 8; k >= 1; k /= 2) top = fmaxf(top, __shfl_xor(top, k));
      scale_for(top, up, down);
      const int block = first / 16 + q;
      if (live && block < blocks) {
        half_t* dst = p.t2 + m * p.ld2 + 32 * block + r;
        split_value<FMT>(t * up, dst[0], dst[16]);
        if (r == 0) p.factor[m * blocks + block] = down * scale;
      }
    }
  }
}

template <int FMT, int RB>
__global__ __launch_bounds__(64 * kWaves) void shrink_kernel(ShrinkArgs p, int64_t base) {
  constexpr int kBytes = XStage<1, 32 * steps_of(RB)>::kBytes;
  static_assert((1 + RB) * kBytes >= RB * 1024, "room for the sums");
  __shared__ __attribute__((aligned(16))) unsigned char lds[kWaves * (1 + RB) * kBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, quarter = lane >> 4;
  const int groups = (p.R + 16 * RB - 1) / (16 * RB);
  const int64_t id = base + blockIdx.x;
  // (a place's blocks of rows one after another: dealt out the other way round,
  // the places that have an adapter would all be on one XCD)
  const int64_t per = ((int64_t)p.M + 15) / 16 * groups, rest = id % per;
  const int slot = (int)(id / per);
  const int first = (int)(rest % groups) * 16 * RB;   // rank
  const int m0 = (int)(rest / groups) * 16;
  const int mine = m0 + r < p.M ? adapter_of(p.ids, m0 + r, p.S) : -1;

  if (slot == 0 && wave == 0 && p.t32) {
    // rows without an adapter: zeros (one that does not exist: NaN)
    for (int q = quarter; q < RB; q += 4)
#pragma unroll 4
      for (int i = 0; i < 16; ++i) {
        const int other = __builtin_amdgcn_readlane(mine, i), c = first + 16 * q + r;
        if (other < 0 && m0 + i < p.M && c < p.R)
          p.t32[(int64_t)(m0 + i) * p.ldt + c] = other == -1 ? 0.f : __builtin_nanf("");
      }
  }
  uint32_t pending = (uint32_t)__ballot(mine >= 0) & 0xFFFFu;
  for (int d = 0; pending; ++d) {
    const int a = __builtin_amdgcn_readlane(mine, __builtin_ctz(pending));
    const uint32_t rows = (uint32_t)__ballot(mine == a) & 0xFFFFu;
    pending &= ~rows;
    if (d % p.slots == slot) {
      if (d >= p.slots) __syncthreads();   // the sums before have been read
      shrink_one<FMT, RB>(p, lds, a, rows, m0, first, lane, wave);
    }
  }
}

template <int FMT>
const void* pick(int rb) {
  return rb == 1   ? (const void*)shrink_kernel<FMT, 1>
         : rb == 2 ? (const void*)shrink_kernel<FMT, 2>
                   : (const void*)shrink_kernel<FMT, 4>;
}

}  // namespace

hipError_t launch_shrink(int fmt, const ShrinkArgs& p, hipStream_t stream) {
  const int rb = p.R <= 16 ? 1 : p.R <= 32 ? 2 : 4;
  const int64_t wgs = ((int64_t)p.M + 15) / 16 * ((p.R + 16 * rb - 1) / (16 * rb));
  ShrinkArgs a = p;
  a.slots = (int)std::max<int64_t>(
      1, std::min<int64_t>(std::min(kMaxSlots, p.M), kWorkgroups / std::max<int64_t>(1, wgs)));
  return launch_tiles(fmt == kFmtBF16 ? pick<kFmtBF16>(rb) : pick<kFmtF16>(rb), a, wgs * a.slots,
                      64 * kWaves, 0, stream);
}

}  // namespace tune
}  // namespace mi355gemm

// C = act(X W^T + bias) + residual with 4-bit weights and group scales, for
// few rows of X: the kernel and its C entry point.
//
// W[n][k] = (q - z) s with one s and z for each group of a row.  A lane takes
// 16 bytes = 32 weights of its row in one load, so a wave takes 16 rows x 128
// k ("a block") at a time.  The nibbles become 16-bit floats without a
// conversion: (word >> 4 i) & 0x000f000f picks k = i and i + 4 of the word's
// eight, and or-ing in an exponent makes 1024 + q (fp16, 0x6400) or 128 + q
// (bf16, 0x4300), both exact.  fp16 then subtracts 1024 + z exactly (packed
// adds); bf16 has no packed add, so a second product of X with ones makes the
// group's sum of x and (128 + z) times it is taken off in fp32 (the matrix
// cores idle here: the bound is HBM).  s multiplies the group's fp32 sum.  X
// is put in the nibbles' order (0 4 1 5 2 6 3 7) in registers.
//
// Where a block holds several groups (a group is a multiple of 32) each step
// of 32 k must lie in one: the four lanes of a row exchange words (a 4 x 4
// transposition by lane-row swaps) so that step j has k = 32 j .. + 31 of the
// block.  Where a block lies in one group the words are used as they come.
#define MI355FUSED_BUILDING 1
#include "skinny.hpp"

namespace mi355gemm {
namespace fused {
namespace {

using namespace skinny;

typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));

constexpr int kBlock = 128;   // K values of a block
constexpr int kUnroll = 4;    // blocks in flight a wave
constexpr int kMaxWaves = 8;

struct W4Args {
  const half_t* X;
  const uint8_t* Wq;
  const half_t* scales;
  const uint8_t* zeros;
  const half_t* bias;
  const half_t* res;
  half_t* C;
  int64_t ldx, ldq, lds, ldz, ldr, ldc;
  int M, N, K, group, act, waves;
};

// How the groups lie in a block: one a block (group % 128 == 0), two of 64,
// four of 32, or any other multiple of 32 (a lookup for each step).
enum Groups { kOne = 0, kTwo, kFour, kAny };

// A block as loaded: weights, and the raw scales and zero points of its
// groups (up to four of each).
struct Block {
  u4 w;
  uint16_t s[4];
  uint8_t z[4];
};

template <int GR, bool TAIL>
__device__ __forceinline__ Block load_block(const W4Args& p, const uint8_t* row,
                                            const half_t* scales, const uint8_t* zeros, int block,
                                            int quarter) {
  Block b;
  const int k0 = block * kBlock;
  const uint8_t* src = row + (int64_t)block * (kBlock / 2) + 16 * quarter;
  if constexpr (!TAIL) {
    __builtin_memcpy(&b.w, src, 16);
  } else {
    // the bytes inside the row only; past it the weights meet zeros of X
    const int have = p.K / 2 + (p.K & 1) - (k0 / 2 + 16 * quarter);
    b.w = u4{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (e < have) b.w[e / 4] |= (uint32_t)src[e] << (8 * (e % 4));
  }
  constexpr int kN = GR == kOne ? 1 : GR == kTwo ? 2 : 4;
  uint16_t s[kN];
  uint8_t z[kN];
  if constexpr (!TAIL && GR != kAny) {
    const int g0 = GR == kOne ? k0 / p.group : block * kN;
    __builtin_memcpy(s, scales + g0, 2 * kN);
    if (zeros) __builtin_memcpy(z, zeros + g0, kN);
  } else {
    // group of each step, the last one past the row's end
    const int last = (p.K - 1) / p.group;
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const int g = min((k0 + j * (kBlock / kN)) / p.group, last);
      s[j] = __builtin_bit_cast(uint16_t, scales[g]);
      if (zeros) z[j] = zeros[g];
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    b.s[j] = s[j * kN / 4];
    b.z[j] = zeros ? z[j * kN / 4] : (uint8_t)8;
  }
  return b;
}

// Word j of lane row c becomes word c of lane row j.
__device__ __forceinline__ u4 transpose4(u4 w) {
  const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u4{c[0], c[1], d[0], d[1]};
}

// Eight nibbles as 16-bit floats 1024 + q (fp16) or 128 + q (bf16), k in the
// order 0 4 1 5 2 6 3 7.
template <int FMT>
__device__ __forceinline__ u4 spread(uint32_t w) {
  constexpr uint32_t kOr = FMT == kFmtF16 ? 0x64006400u : 0x43004300u;
  return u4{(w & 0x000f000fu) | kOr, ((w >> 4) & 0x000f000fu) | kOr,
            ((w >> 8) & 0x000f000fu) | kOr, ((w >> 12) & 0x000f000fu) | kOr};
}

// The same order for eight X values.
__device__ __forceinline__ h8 reorder(h8 v) {
  return __builtin_shufflevector(v, v, 0, 4, 1, 5, 2, 6, 3, 7);
}

template <int FMT, int GR, int MT, bool TAIL>
__device__ __forceinline__ void multiply(const W4Args& p, const Block& b,
                                         const half_t* const (&xrow)[MT], int block, int quarter,
                                         f4 (&tot)[MT]) {
  const u4 w = GR == kOne ? b.w : transpose4(b.w);
  f4 acc[MT], sum[MT];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    constexpr int kSteps = GR == kOne ? 4 : GR == kTwo ? 2 : 1;   // steps of a group
    if (j % kSteps == 0) {
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[t] = sum[t] = f4{0.f, 0.f, 0.f, 0.f};
    }
    const int k = block * kBlock + (GR == kOne ? 32 * quarter + 8 * j : 32 * j + 8 * quarter);
    u4 q = spread<FMT>(w[j]);
    if constexpr (FMT == kFmtF16) {
      const half_t off = (half_t)(-1024.f - (float)b.z[j]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t pair = q[i];
        q[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(h2, pair) + h2{off, off});
      }
    }
    const h8 wf = __builtin_bit_cast(h8, q);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const h8 x = reorder(load_x<TAIL>(xrow[t], k, p.K));
      acc[t] = mfma16<FMT>(x, wf, acc[t]);
      if constexpr (FMT == kFmtBF16) {
        const u4 ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
        sum[t] = mfma16<FMT>(x, __builtin_bit_cast(h8, ones), sum[t]);
      }
    }
    if (j % kSteps == kSteps - 1) {
      const float s = word_to_f32<FMT>(__builtin_bit_cast(half_t, b.s[j]));
      const float off = 128.f + (float)b.z[j];
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          tot[t][v] += s * (FMT == kFmtBF16 ? acc[t][v] - off * sum[t][v] : acc[t][v]);
    }
  }
}

template <int FMT, int GR, int MT>
__global__ __launch_bounds__(64 * kMaxWaves) void w4_kernel(W4Args p, int64_t base) {
  extern __shared__ __attribute__((aligned(16))) float lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, quarter = lane >> 4;
  const int64_t groups_n = (p.N + 15) / 16;
  const int64_t id = base + blockIdx.x;
  const int m0 = (int)(id / groups_n) * 64;
  const int n = (int)(id % groups_n) * 16 + r;
  const int row = n < p.N ? n : p.N - 1;   // rows past N repeat the last one, unstored
  const uint8_t* wrow = p.Wq + row * p.ldq;
  const half_t* scales = p.scales + row * p.lds;
  const uint8_t* zeros = p.zeros ? p.zeros + row * p.ldz : nullptr;
  const half_t* xrow[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int m = m0 + 16 * t + r;
    xrow[t] = p.X + (m < p.M ? m : p.M - 1) * p.ldx;   // rows past M repeat the last, unstored
  }
  f4 tot[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) tot[t] = f4{0.f, 0.f, 0.f, 0.f};

  // chunks of kUnroll blocks, in turn to the waves; then the blocks left over
  const int full = p.K / kBlock, chunks = full / kUnroll;
  Block cur[kUnroll], nxt[kUnroll];
  int c = wave;
  if (c < chunks) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      cur[u] = load_block<GR, false>(p, wrow, scales, zeros, c * kUnroll + u, quarter);
  }
  for (; c < chunks; c += p.waves) {
    const int cn = c + p.waves < chunks ? c + p.waves : c;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      nxt[u] = load_block<GR, false>(p, wrow, scales, zeros, cn * kUnroll + u, quarter);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      multiply<FMT, GR, MT, false>(p, cur[u], xrow, c * kUnroll + u, quarter, tot);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) cur[u] = nxt[u];
  }
  const int left = chunks * kUnroll;
  for (int b = left + wave; b < full; b += p.waves) {
    const Block k = load_block<GR, false>(p, wrow, scales, zeros, b, quarter);
    multiply<FMT, GR, MT, false>(p, k, xrow, b, quarter, tot);
  }
  if (full * kBlock < p.K && wave == (full - left) % p.waves) {
    const Block k = load_block<GR, true>(p, wrow, scales, zeros, full, quarter);
    multiply<FMT, GR, MT, true>(p, k, xrow, full, quarter, tot);
  }

  add_waves<MT>(tot, lds, wave, lane, p.waves);
  if (wave > 0 || n >= p.N) return;
  const float bias = p.bias ? word_to_f32<FMT>(p.bias[n]) : 0.f;
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int m = m0 + 16 * t + 4 * quarter + v;
      if (m >= p.M) continue;
      float y = epi_act(tot[t][v] + bias, p.act);
      if (p.res) y += word_to_f32<FMT>(p.res[m * p.ldr + n]);
      p.C[m * p.ldc + n] = f32_to_word<FMT>(y);
    }
}

typedef void (*W4Kernel)(W4Args, int64_t);

template <int FMT, int GR>
W4Kernel pick_rows(int M) {
  return M <= 16 ? w4_kernel<FMT, GR, 1> : M <= 32 ? w4_kernel<FMT, GR, 2> : w4_kernel<FMT, GR, 4>;
}

template <int FMT>
W4Kernel pick(int M, int group) {
  if (group % kBlock == 0) return pick_rows<FMT, kOne>(M);
  if (group == 64) return pick_rows<FMT, kTwo>(M);
  if (group == 32) return pick_rows<FMT, kFour>(M);
  return pick_rows<FMT, kAny>(M);
}

}  // namespace
}  // namespace fused
}  // namespace mi355gemm

using namespace mi355gemm;
using namespace mi355gemm::fused;

extern "C" MI355FUSED_API int gemm_w4(int type, int M, int N, int K, int group, const void* X,
                                      int ldx, const void* Wq, int ldq, const void* scales, int lds,
                                      const void* zeros, int ldz, const void* bias, int act,
                                      const void* residual, int ldr, void* C, int ldc,
                                      void* stream) {
  if (M < 0 || N < 0 || K < 0) return GEMM_ERR_NEGATIVE_DIM;
  if (bad_type(type) || bad_act(act) || group <= 0 || group % 32 != 0) return GEMM_ERR_BAD_ARG;
  if (M == 0 || N == 0) return GEMM_OK;
  const int64_t groups = ((int64_t)K + group - 1) / group;
  if (bad_ld(ldx, K) || bad_ld(ldq, ((int64_t)K + 1) / 2) || bad_ld(lds, groups) ||
      (zeros && bad_ld(ldz, groups)) || (residual && bad_ld(ldr, N)) || bad_ld(ldc, N))
    return GEMM_ERR_BAD_LD;
  if (C == nullptr || (K > 0 && (X == nullptr || Wq == nullptr || scales == nullptr)))
    return GEMM_ERR_NULL_POINTER;
  const int cus = check_device();
  if (cus < 0) return cus;
  W4Args a{static_cast<const half_t*>(X), static_cast<const uint8_t*>(Wq),
           static_cast<const half_t*>(scales), static_cast<const uint8_t*>(zeros),
           static_cast<const half_t*>(bias), static_cast<const half_t*>(residual),
           static_cast<half_t*>(C), ldx, ldq, lds, ldz, ldr, ldc, M, N, K, group, act, 0};
  const int mt = M <= 16 ? 1 : M <= 32 ? 2 : 4;
  const int64_t wgs = ((int64_t)N + 15) / 16 * (((int64_t)M + 63) / 64);
  const int waves = skinny::waves_for(wgs, std::max(1, K / kBlock), kMaxWaves, cus);
  a.waves = waves;
  const unsigned lds_bytes = (unsigned)((waves - 1) * mt * 64 * sizeof(f4));
  const void* k = type == GEMM_TYPE_BF16 ? (const void*)pick<kFmtBF16>(M, group)
                                         : (const void*)pick<kFmtF16>(M, group);
  return to_status(launch_tiles(k, a, wgs, 64 * waves, lds_bytes, static_cast<hipStream_t>(stream)));
}

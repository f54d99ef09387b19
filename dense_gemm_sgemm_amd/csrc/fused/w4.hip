// C = act(X W^T + bias) + residual with 4-bit weights and group scales, for
// few rows of X: the kernel and its C entry point.
//
// W[n][k] = (q - z) s with one s and z for each group of a row.  A lane takes
// 16 bytes = 32 weights of its row in one load, so a wave takes 16 rows x 128
// k ("a block") at a time.  The nibbles become 16-bit floats without a
// conversion: a mask picks k = i and i + 4 of a word's eight, and or-ing in an
// exponent makes 1024 + q or 64 + q (fp16) or 128 + q (bf16), all exact.  fp16
// then subtracts the offset and z exactly (packed adds); bf16 has no packed
// add, so a second product of X with ones makes the group's sum of x and
// (128 + z) times it is taken off in fp32 (the matrix cores idle here: the
// bound is HBM).  s multiplies the group's fp32 sum.  X is put in the nibbles'
// order (0 4 1 5 2 6 3 7), once where it is kept in LDS.  Where an x of bf16 is
// infinite, or so large (from 2^120) that the two sums overflow, their
// difference is NaN or infinite: such outputs, and no others, are computed
// again from the weights q - z themselves (multiply_exact), so that they are
// what the definition gives.
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
// How the groups lie in blocks: one a block (128), two (64), four (32), one
// for several blocks (a larger multiple of 128: looked up for each block), or
// any other multiple of 32 (looked up for each step of 32 k).
enum Groups { kOne = 0, kTwo, kFour, kWide, kAny };
constexpr int groups_per_block(int gr) { return gr == kTwo ? 2 : gr >= kFour && gr != kWide ? 4 : 1; }
inline int groups_of(int group) {
  return group == kBlock ? kOne : group == 64 ? kTwo : group == 32 ? kFour
         : group % kBlock == 0 ? kWide : kAny;
}

// Blocks of a chunk (a wave has two chunks in flight): four; two where each
// block brings four groups' scales or four blocks of X rows, one where both:
// more registers would spill (64 x 4096 x 16384: 64.9 against 35.5 us); two
// for up to 16 rows in bf16 with two groups a block, whose 170 registers leave
// a SIMD too few waves (16 x 10000 x 2432: 10.6 against 8.7 us; not fp16's 130:
// 8.4 against 8.9); two with sixteen waves.  Two instances still spill: bf16
// with 17 to 32 rows and groups of 64 (6 registers) or of other multiples of 32
// (26).  Half the blocks end that, but not for the better everywhere, by shape:
// 24 x 16384 x 4096 27.9 against 33.5 us, 24 x 4096 x 16384 27.5 against 27.4,
// 32 x 4096 x 4096 10.5 against 9.4 (groups of 64); 50.7 against 56.2, 43.2
// against 36.1 and 19.4 against 15.2 (groups of 96).
constexpr int unroll_of(int fmt, int gr, int mt, int most) {
  const bool four = groups_per_block(gr) == 4;
  if (four && mt == 4) return 1;
  if (four || mt == 4 || most == 16) return 2;
  return mt == 1 && gr == kTwo && fmt == kFmtBF16 ? 2 : 4;
}
// The most waves of a workgroup: four with four blocks of X rows (two
// workgroups' LDS a CU), eight, or sixteen: with X in LDS where chunks are two
// blocks and the registers of sixteen waves do (1 x 4096 x 16384, groups of 32:
// 15.0 against 13.0 us); with X staged and up to 16 rows where a CU has one
// workgroup and each wave four chunks (bf16 with groups of 32 would spill: 19.1
// against 27.7).  Eight against sixteen waves with X staged, 4 and 16 rows, 4096
// weight rows out of HBM, us:
//             K = 8192               K = 11008              K = 16384
//   fp16 128  11.0  11.0  11.5 11.4  14.2 11.6  14.9 12.8   17.5 17.1  18.5 19.1
//   fp16  64  11.1  11.3  11.4 11.7  14.4 12.3  14.9 13.7   18.1 17.7  18.6 19.6
//   fp16  32  12.4  11.8  12.5 12.2  14.1 13.1  14.8 14.5   20.1 18.4  20.7 20.0
//   bf16 128  11.9  11.3  12.6 11.5  15.0 11.9  16.3 12.9   18.8 17.7  20.2 19.2
//   bf16  64  12.0  11.3  12.1 11.9  13.3 12.3  14.5 14.0   19.3 17.8  19.7 19.7
// so the rule loses up to 5 % in fp16 at 16 rows, and two chunks a wave (K from
// 8192) would do in most of the other cases.
constexpr int x_waves(int fmt, int gr) {
  return gr == kFour || (gr == kTwo && fmt == kFmtBF16) ? 16 : 8;
}
constexpr bool sixteen_staged(int fmt, int gr) {
  return gr == kOne || gr == kTwo || (gr == kFour && fmt == kFmtF16);
}
// The threads that registers are allotted for.  Four waves may have 512 each:
// bf16 with four blocks of X rows and several groups a block spills in 256 (64
// x 4096 x 16384, groups of 64: 65.4 against 41.0 us); the others do not, and a
// CU holds two workgroups of them (64 x 16384 x 4096 fp16, groups of 32: 40.8
// against 57.8 us in more than 256).
constexpr int bound_of(int fmt, int gr, int mt, int most) {
  return 64 * (mt == 4 && (fmt == kFmtF16 || groups_per_block(gr) == 1) ? 8 : most);
}
constexpr int kStaged = 4;    // 16-byte pieces of X a thread loads ahead of its weights
// X of up to three rows is kept in LDS where it takes no more than kXBytes, or,
// with a workgroup a CU at most, kXBytesAlone; with more rows each wave's own
// copy is no slower, and smaller (1 x 4096 x 16384: 12.1 against 16.4 us in
// LDS; 3 x 16384 x 4096: 12.7 against 14.3; 5 x 16384 x 4096: 17.0 against 14.5).
constexpr int kXRows = 3, kXBytes = 32 << 10, kXBytesAlone = 56 << 10;
constexpr int kXBytesSixteen = 48 << 10;   // beside sixteen waves' sums

struct W4Args {
  const half_t* X;
  const uint8_t* Wq;
  const half_t* scales;
  const uint8_t* zeros;
  const half_t* bias;
  const half_t* res;
  half_t* C;
  int64_t ldx, ldq, lds, ldz, ldr, ldc;
  int M, N, K, group, act, waves, chunks;
};

// U blocks as loaded: weights, and the raw scales and zero points of their groups.
template <int GR, int U>
struct Blocks {
  static constexpr int kG = groups_per_block(GR);
  u4 w[U];
  uint16_t s[U * kG];
  uint8_t z[U * kG];
};

// A pointer to global memory: loads through it are no flat loads, which would
// wait for LDS reads too.
template <typename T>
using Global = __attribute__((address_space(1))) const T*;

// Zero points of a call without any.
__device__ const uint8_t kEights[16] = {8, 8, 8, 8, 8, 8, 8, 8, 8, 8, 8, 8, 8, 8, 8, 8};

// A lane's weight row.  No zero points: kEights, whose groups all have index 0.
struct Row {
  Global<uint8_t> w;
  Global<uint16_t> s;
  Global<uint8_t> z;
  int z_mask;
};

template <int GR, int U, bool TAIL>
__device__ __forceinline__ void load_blocks(const W4Args& p, const Row& row, int block, int quarter,
                                            Blocks<GR, U>& b) {
  constexpr int kG = Blocks<GR, U>::kG;
  const int k0 = block * kBlock;
  Global<uint8_t> src = row.w + (int64_t)block * (kBlock / 2) + 16 * quarter;
  if constexpr (!TAIL) {
#pragma unroll
    for (int u = 0; u < U; ++u) __builtin_memcpy(&b.w[u], src + u * (kBlock / 2), 16);
  } else {
    // one block: the bytes inside the row only; past it the weights meet zeros of X
    const int have = p.K / 2 + (p.K & 1) - (k0 / 2 + 16 * quarter);
    u4 w = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (e < have) w[e / 4] |= (uint32_t)src[e] << (8 * (e % 4));
    b.w[0] = w;
  }
  if constexpr (!TAIL && GR <= kFour) {
    const int g0 = block * kG;
    __builtin_memcpy(b.s, row.s + g0, 2 * U * kG);
    __builtin_memcpy(b.z, row.z + (g0 & row.z_mask), U * kG);
  } else {
    // the group of each block or step, the last one past the row's end
    const int last = (p.K - 1) / p.group;
#pragma unroll
    for (int j = 0; j < U * kG; ++j) {
      const int g = min((k0 + j * (kBlock / kG)) / p.group, last);
      b.s[j] = row.s[g];
      b.z[j] = row.z[g & row.z_mask];
    }
  }
}

// Word j of lane row c becomes word c of lane row j.
__device__ __forceinline__ u4 transpose4(u4 w) {
  const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u4{c[0], c[1], d[0], d[1]};
}

// a & mask | bits in one instruction: the two constants would not both fit it
// as literals, so `bits` is kept in a register the compiler cannot see through.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t bits) {
  return (a & mask) | bits;
}
template <int FMT>
struct Magic {
  uint32_t low, high;
  __device__ __forceinline__ Magic() {
    low = FMT == kFmtF16 ? 0x64006400u : 0x43004300u;
    high = 0x54005400u;
    asm("" : "+v"(low));
    if constexpr (FMT == kFmtF16) asm("" : "+v"(high));
  }
};

// Eight nibbles as 16-bit floats, k in the order 0 4 1 5 2 6 3 7: bf16 128 + q;
// fp16 q - z, from 1024 + q where the nibble lies in the low four bits of a
// half word and 64 + q where it lies in the next four (no shift).
template <int FMT>
__device__ __forceinline__ u4 spread(uint32_t w, const Magic<FMT>& magic, float z) {
  if constexpr (FMT == kFmtF16) {
    const half_t a = (half_t)(-1024.f - z), b = (half_t)(-64.f - z);
    const h2 offa = {a, a}, offb = {b, b};
    const uint32_t v = w >> 8;
    const uint32_t q[4] = {and_or(w, 0x000f000fu, magic.low), and_or(w, 0x00f000f0u, magic.high),
                           and_or(v, 0x000f000fu, magic.low), and_or(v, 0x00f000f0u, magic.high)};
    u4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(h2, q[i]) + (i & 1 ? offb : offa));
    return r;
  } else {
    return u4{and_or(w, 0x000f000fu, magic.low), and_or(w >> 4, 0x000f000fu, magic.low),
              and_or(w >> 8, 0x000f000fu, magic.low), and_or(w >> 12, 0x000f000fu, magic.low)};
  }
}

// The same order for eight X values.
__device__ __forceinline__ h8 reorder(h8 v) {
  return __builtin_shufflevector(v, v, 0, 4, 1, 5, 2, 6, 3, 7);
}

// First k of step j of a block for a lane.
template <int GR>
__device__ __forceinline__ int step_k(int j, int quarter) {
  return groups_per_block(GR) == 1 ? 32 * quarter + 8 * j : 32 * j + 8 * quarter;
}

// One block's products.  x[t][j]: the X fragments of its four steps, reordered.
template <int FMT, int GR, int MT>
__device__ __forceinline__ void multiply(u4 raw, const uint16_t* scales, const uint8_t* zeros,
                                         const h8 (&x)[MT][4], const Magic<FMT>& magic,
                                         f4 (&tot)[MT]) {
  constexpr int kG = groups_per_block(GR), kSteps = 4 / kG;   // steps of a group
  const u4 w = kG == 1 ? raw : transpose4(raw);
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    f4 acc[MT], sum[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = sum[t] = f4{0.f, 0.f, 0.f, 0.f};
    const float z = (float)zeros[g];
#pragma unroll
    for (int j = g * kSteps; j < (g + 1) * kSteps; ++j) {
      const h8 wf = __builtin_bit_cast(h8, spread<FMT>(w[j], magic, z));
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        acc[t] = mfma16<FMT>(x[t][j], wf, acc[t]);
        if constexpr (FMT == kFmtBF16) {
          const u4 ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
          sum[t] = mfma16<FMT>(x[t][j], __builtin_bit_cast(h8, ones), sum[t]);
        }
      }
    }
    const uint16_t bits = scales[g];
    const float s = word_to_f32<FMT>(__builtin_bit_cast(half_t, bits));
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        tot[t][v] += s * (FMT == kFmtBF16 ? acc[t][v] - (128.f + z) * sum[t][v] : acc[t][v]);
  }
}

// One block's products in bf16 with the weights q - z themselves, times 2^-12: a
// group's sum of 128 products of up to 15 x 2^128 stays finite, and so the
// result, 2^-12 of tot, is infinite or NaN only where the definition's is (or
// where it is infinite within a factor of 2^12 and cancels later).
template <int GR, int MT>
__device__ __forceinline__ void multiply_exact(u4 raw, const uint16_t* scales, const uint8_t* zeros,
                                               const h8 (&x)[MT][4], f4 (&tot)[MT]) {
  constexpr int kG = groups_per_block(GR), kSteps = 4 / kG;
  const u4 w = kG == 1 ? raw : transpose4(raw);
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    f4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = g * kSteps; j < (g + 1) * kSteps; ++j) {
      // the nibbles' order of spread; differences of at most 15 are exact
      auto word = [&](int nibble) __attribute__((always_inline)) {
        const int q = (w[j] >> (4 * nibble)) & 15;
        return __float_as_uint((float)(q - (int)zeros[g]) * 0x1p-12f) >> 16;
      };
      u4 r;
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = word(i) | (word(i + 4) << 16);
#pragma unroll
      for (int t = 0; t < MT; ++t)
        acc[t] = mfma16<kFmtBF16>(x[t][j], __builtin_bit_cast(h8, r), acc[t]);
    }
    const uint16_t bits = scales[g];
    const float s = word_to_f32<kFmtBF16>(__builtin_bit_cast(half_t, bits));
#pragma unroll
    for (int t = 0; t < MT; ++t) tot[t] += s * acc[t];
  }
}

// XL: the rows of X (M <= 16) lie in LDS, reordered, zero past K, in
// rows of K rounded up to blocks plus 16 bytes (rows then start in different
// banks).  Otherwise each wave stages the rows of a block in turn (XStage).
template <int FMT, int GR, int MT, bool XL, int MOST>
__global__ __launch_bounds__(bound_of(FMT, GR, MT, MOST)) void w4_kernel(W4Args p, int64_t base) {
  constexpr int kUnroll = unroll_of(FMT, GR, MT, XL ? 8 : MOST);
  typedef XStage<MT, kBlock> Stage;
  extern __shared__ __attribute__((aligned(16))) unsigned char dynamic_lds[];
  __shared__ __attribute__((aligned(16))) unsigned char
      stage_lds[XL ? 16 : MOST * Stage::kBytes];
  unsigned char* lds = XL ? dynamic_lds : stage_lds;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, quarter = lane >> 4;
  const int64_t groups_n = (p.N + 15) / 16;
  const int64_t id = base + blockIdx.x;
  const int m0 = (int)(id / groups_n) * 64;
  const int n = (int)(id % groups_n) * 16 + r;
  const int nr = n < p.N ? n : p.N - 1;   // rows past N repeat the last one, unstored
  const Row row{(Global<uint8_t>)(p.Wq + nr * p.ldq), (Global<uint16_t>)(p.scales + nr * p.lds),
                p.zeros ? (Global<uint8_t>)(p.zeros + nr * p.ldz) : (Global<uint8_t>)kEights,
                p.zeros ? -1 : 0};
  const int blocks = (int)(((int64_t)p.K + kBlock - 1) / kBlock), full = p.K / kBlock;
  const int64_t x_pitch = (int64_t)blocks * (kBlock * 2) + 16;

  // X's first pieces, then the wave's first two chunks of weights, then the
  // pieces go to LDS: loads return in order, so X does not wait for them.
  h8 staged[kStaged];
  const int row_pieces = blocks * (kBlock / 8);
  const int pieces = p.M * row_pieces;
  auto load_piece = [&](int i) __attribute__((always_inline)) {
    return reorder(load_x<true>(p.X + (int64_t)(i / row_pieces) * p.ldx, i % row_pieces * 8, p.K));
  };
  auto store_piece = [&](int i, h8 v) __attribute__((always_inline)) {
    *(h8*)(lds + i / row_pieces * x_pitch + i % row_pieces * 16) = v;
  };
  if constexpr (XL) {
#pragma unroll
    for (int q = 0; q < kStaged; ++q)
      if (tid + q * (int)blockDim.x < pieces) staged[q] = load_piece(tid + q * blockDim.x);
    __builtin_amdgcn_sched_barrier(0);
  }
  Blocks<GR, kUnroll> cur, nxt;
  int c = wave;
  if (c < p.chunks) {
    load_blocks<GR, kUnroll, false>(p, row, c * kUnroll, quarter, cur);
    if (c + p.waves < p.chunks)
      load_blocks<GR, kUnroll, false>(p, row, (c + p.waves) * kUnroll, quarter, nxt);
  }
  if constexpr (XL) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < kStaged; ++q)
      if (tid + q * (int)blockDim.x < pieces) store_piece(tid + q * blockDim.x, staged[q]);
    for (int i = tid + kStaged * blockDim.x; i < pieces; i += blockDim.x)
      store_piece(i, load_piece(i));
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  }

  // Fragments of X (rows past M repeat the last one, unstored).
  const unsigned char* xl = lds + (r < p.M ? r : p.M - 1) * x_pitch;
  unsigned char* buf = lds + wave * Stage::kBytes;
  Stage stage;
  auto read_x = [&](h8 (&x)[MT][4], int block) __attribute__((always_inline)) {
    if constexpr (!XL) stage.store(buf, lane, [](h8 v) { return reorder(v); });
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = step_k<GR>(j, quarter);
        x[t][j] = XL ? *(const h8*)(xl + 2 * (block * kBlock + k)) : Stage::read(buf, t, r, k);
      }
  };
  auto load_rows = [&](int block, auto tail) __attribute__((always_inline)) {
    if constexpr (!XL)
      stage.template load<decltype(tail)::value>(p.X, p.ldx, m0, p.M, block * kBlock, p.K, lane);
  };
  constexpr int kG = groups_per_block(GR);
  const Magic<FMT> magic;
  f4 tot[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) tot[t] = f4{0.f, 0.f, 0.f, 0.f};

  const std::integral_constant<bool, false> inside{};
  const std::integral_constant<bool, true> at_end{};
  h8 x[MT][4];
  if (c < p.chunks) load_rows(c * kUnroll, inside);
  for (; c < p.chunks; c += p.waves) {
    const int cn = c + p.waves < p.chunks ? c + p.waves : c;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      read_x(x, c * kUnroll + u);
      load_rows(u + 1 < kUnroll ? c * kUnroll + u + 1 : cn * kUnroll, inside);
      multiply<FMT, GR, MT>(cur.w[u], cur.s + u * kG, cur.z + u * kG, x, magic, tot);
    }
    cur = nxt;
    if (c + 2 * p.waves < p.chunks)
      load_blocks<GR, kUnroll, false>(p, row, (c + 2 * p.waves) * kUnroll, quarter, nxt);
  }
  // blocks left over, one at a time in turn to the waves
  const int left = p.chunks * kUnroll;
  Blocks<GR, 1> one;
  for (int b = left + wave; b < full; b += p.waves) {
    load_blocks<GR, 1, false>(p, row, b, quarter, one);
    load_rows(b, inside);
    read_x(x, b);
    multiply<FMT, GR, MT>(one.w[0], one.s, one.z, x, magic, tot);
  }
  if (full < blocks && wave == (full - left) % p.waves) {
    load_blocks<GR, 1, true>(p, row, full, quarter, one);
    load_rows(full, at_end);
    read_x(x, full);
    multiply<FMT, GR, MT>(one.w[0], one.s, one.z, x, magic, tot);
  }

  if constexpr (FMT == kFmtBF16) {
    // Sums that are no numbers, again and exactly.  Once infinite or NaN a sum
    // stays so, and each of them is mended by itself: a row's outputs do not
    // depend on the other rows.
    auto lost = [](float v) { return !(fabsf(v) < __builtin_inff()); };
    bool any = false;
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v) any |= lost(tot[t][v]);
    if (__ballot(any) != 0) {
      f4 again[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) again[t] = f4{0.f, 0.f, 0.f, 0.f};
      auto block = [&](int b, auto tail) __attribute__((always_inline)) {
        load_blocks<GR, 1, decltype(tail)::value>(p, row, b, quarter, one);
        load_rows(b, tail);
        read_x(x, b);
        multiply_exact<GR, MT>(one.w[0], one.s, one.z, x, again);
      };
      // the wave's blocks: its chunks and what was left over
      const int mine = p.chunks > wave ? (p.chunks - wave + p.waves - 1) / p.waves * kUnroll : 0;
#pragma unroll 1
      for (int i = 0; i < mine; ++i)
        block((wave + i / kUnroll * p.waves) * kUnroll + i % kUnroll, inside);
#pragma unroll 1
      for (int b = left + wave; b < full; b += p.waves) block(b, inside);
      if (full < blocks && wave == (full - left) % p.waves) block(full, at_end);
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (lost(tot[t][v])) tot[t][v] = again[t][v] * 0x1p12f;
    }
  }

  // (the sums take the place of X)
  if (!XL) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  add_waves<MT>(tot, reinterpret_cast<float*>(lds + (XL ? p.M * x_pitch : 0)), wave, lane, p.waves);
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

template <int FMT, int GR>
const void* pick_rows(int M, bool x_in_lds, int most) {
  if (x_in_lds) return (const void*)w4_kernel<FMT, GR, 1, true, x_waves(FMT, GR)>;
  if constexpr (sixteen_staged(FMT, GR))
    if (most == 16) return (const void*)w4_kernel<FMT, GR, 1, false, 16>;
  return M <= 16   ? (const void*)w4_kernel<FMT, GR, 1, false, 8>
         : M <= 32 ? (const void*)w4_kernel<FMT, GR, 2, false, 8>
                   : (const void*)w4_kernel<FMT, GR, 4, false, 4>;
}

template <int FMT>
const void* pick(int M, int gr, bool x_in_lds, int most) {
  switch (gr) {
    case kOne: return pick_rows<FMT, kOne>(M, x_in_lds, most);
    case kTwo: return pick_rows<FMT, kTwo>(M, x_in_lds, most);
    case kFour: return pick_rows<FMT, kFour>(M, x_in_lds, most);
    case kWide: return pick_rows<FMT, kWide>(M, x_in_lds, most);
    default: return pick_rows<FMT, kAny>(M, x_in_lds, most);
  }
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
  const int status = check_sizes(M, N, K);
  if (status != GEMM_OK) return status;
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
           static_cast<half_t*>(C), ldx, ldq, lds, ldz, ldr, ldc, M, N, K, group, act, 0, 0};
  const int mt = M <= 16 ? 1 : M <= 32 ? 2 : 4;
  const int64_t wgs = ((int64_t)N + 15) / 16 * (((int64_t)M + 63) / 64);
  const int64_t blocks = ((int64_t)K + kBlock - 1) / kBlock;
  const int64_t x_bytes = M * (blocks * kBlock * 2 + 16);
  const bool x_in_lds =
      M <= kXRows && K > 0 && x_bytes <= (wgs <= cus ? kXBytesAlone : kXBytes);
  const int fmt = type == GEMM_TYPE_BF16 ? kFmtBF16 : kFmtF16, gr = groups_of(group);
  int most = mt == 4 ? 4 : 8;
  if (x_in_lds)
    most = x_bytes <= kXBytesSixteen ? x_waves(fmt, gr) : 8;
  else if (mt == 1 && sixteen_staged(fmt, gr) && wgs <= cus && blocks >= 4 * 16 * 2)
    most = 16;
  // whole chunks where four waves have one each, else single blocks
  const int unroll = unroll_of(fmt, gr, mt, x_in_lds ? 8 : most);
  a.chunks = K / kBlock >= 4 * unroll ? K / (kBlock * unroll) : 0;
  a.waves = skinny::waves_for(wgs, a.chunks ? a.chunks : std::max<int>(1, (int)blocks), most, cus);
  const unsigned lds_bytes =
      x_in_lds ? (unsigned)(x_bytes + (a.waves - 1) * mt * 64 * sizeof(f4)) : 0;
  const void* k = fmt == kFmtBF16 ? pick<kFmtBF16>(M, gr, x_in_lds, most)
                                  : pick<kFmtF16>(M, gr, x_in_lds, most);
  return to_status(
      launch_tiles(k, a, wgs, 64 * a.waves, lds_bytes, static_cast<hipStream_t>(stream)));
}

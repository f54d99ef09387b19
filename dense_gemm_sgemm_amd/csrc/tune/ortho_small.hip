// gemm_ortho for matrices whose shorter side s is at most 64 (an adapter's
// factors): every product is tiny, and what counts is the number of launches
// that wait for each other.  One launch a step: a workgroup takes a slab of the
// longer side, adds up the slabs' parts of A = X X^T that the launch before
// left, makes C = a I + b A + c A^2 in LDS (every workgroup for itself), its slab
// of C X, and the slab's part of the next A.
//
// X is kept as its columns, [t][SP] with SP = 32 or 64, so that a fragment of
// either operand is 16 bytes in a row; A and C are symmetric.  Everything is in
// two binary16 values, hi + lo, with the powers of two of ortho.hip, and each
// product is hi hi + hi lo + lo hi: the matrix cores are idle anyway.  Sixteen
// 16 x 4096: 8.9 us a step (its launch, one latency for X and one for the parts of
// A), 12 for the first iterate.
//
// The slab is multiplied both ways round.  X^T C leaves a lane four columns of
// one row of the result, and those of two blocks of 16 columns are, as they
// stand, a fragment of the next A's product over columns (any order of the summed
// index will do if both operands have the same).  C X leaves it four rows of
// one column, which is how X is stored.
#include "ortho.hpp"

namespace mi355gemm {
namespace tune {
namespace ortho {
namespace {

using hgemm::f4;
using hgemm::h4;
constexpr int kWaves = kThreads / 64, kCols = 32;   // columns a wave takes at a time

struct SmallArgs {
  StartArgs st;
  const half_t* from[2];   // hi, lo of the iterate, [L][columns][SP]
  half_t* to[2];
  const float* gram;       // its A in parts, [L][slabs][SP][SP]
  float* gram_to;
  int slabs, slab, steps;
  float alpha, beta, gamma;
  hgemm::Growth growth;
  int last;
  SmallOut out;
};

__device__ __forceinline__ f4 mul(h8 a, h8 b, f4 c) { return hgemm::mfma16<kFmtF16>(a, b, c); }

__device__ __forceinline__ void split4(f4 v, h4& hi, h4& lo) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    hi[e] = (half_t)v[e];
    lo[e] = (half_t)(v[e] - (float)hi[e]);
  }
}

// The blocks (i, j), j <= i, of the products of 32 columns' fragments.
template <int NB>
__device__ __forceinline__ void add_gram(const h8 (&hi)[NB], const h8 (&lo)[NB],
                                         f4 (&acc)[NB * (NB + 1) / 2]) {
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j <= i; ++j) {
      f4& a = acc[i * (i + 1) / 2 + j];
      a = mul(hi[i], hi[j], a);
      a = mul(hi[i], lo[j], a);
      a = mul(lo[i], hi[j], a);
    }
}

// The waves' sums, added up and stored on both sides of the diagonal.
template <int SP>
__device__ __forceinline__ void store_gram(f4 (&acc)[SP / 16 * (SP / 16 + 1) / 2], f4* lds,
                                           float* dst, int wave, int lane) {
  constexpr int NB = SP / 16, kBlocks = NB * (NB + 1) / 2;
  __syncthreads();
  if (wave > 0) {
#pragma unroll
    for (int q = 0; q < kBlocks; ++q) lds[((wave - 1) * kBlocks + q) * 64 + lane] = acc[q];
  }
  __syncthreads();
  if (wave > 0) return;
  const int g = lane >> 4, r = lane & 15;
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j <= i; ++j) {
      const int q = i * (i + 1) / 2 + j;
      for (int w = 0; w + 1 < kWaves; ++w) acc[q] += lds[(w * kBlocks + q) * 64 + lane];
      // rows 16 i + 4 g + v, column 16 j + r
#pragma unroll
      for (int v = 0; v < 4; ++v) dst[(16 * i + 4 * g + v) * SP + 16 * j + r] = acc[q][v];
      if (i != j) *(f4*)(dst + (16 * j + r) * SP + 16 * i + 4 * g) = acc[q];
    }
}

// X0 and its part of A.
template <int SP>
__global__ __launch_bounds__(kThreads) void small_start_kernel(SmallArgs p, int64_t base) {
  constexpr int NB = SP / 16, kBlocks = NB * (NB + 1) / 2;
  __shared__ f4 lds[(kWaves - 1) * kBlocks * 64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int64_t id = base + blockIdx.x, l = id / p.slabs;
  const int slab = (int)(id % p.slabs);
  const StartArgs& st = p.st;
  const bool tall = st.m > st.n;
  const int s = tall ? st.n : st.m, t = tall ? st.m : st.n;
  double up, rho;
  start_of(st, l, up, rho);
  if (slab == 0 && threadIdx.x == 0) put_coef(st, l, rho);
  const char* G = static_cast<const char*>(st.G) + l * st.stride_g * (st.type == kF32 ? 4 : 2);
  f4 acc[kBlocks];
#pragma unroll
  for (int q = 0; q < kBlocks; ++q) acc[q] = f4{0.f, 0.f, 0.f, 0.f};
  const int64_t columns = (int64_t)p.slabs * p.slab;
  for (int c = wave * kCols; c < p.slab; c += kWaves * kCols) {
    const int n0 = slab * p.slab + c;
    h8 hi[NB], lo[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int row = 16 * i + r;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        f4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int n = n0 + 16 * b + 4 * g + e;
          const int64_t at = tall ? (int64_t)n * st.ldg + row : (int64_t)row * st.ldg + n;
          const float x = row < s && n < t ? load_one(G, at, st.type) : 0.f;
          v[e] = (float)((double)x * up);
        }
        h4 h, w;
        split4(v, h, w);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t at = (l * columns + n0 + 16 * b + 4 * g + e) * SP + row;
          p.to[0][at] = h[e];
          p.to[1][at] = w[e];
          hi[i][4 * b + e] = h[e];
          lo[i][4 * b + e] = w[e];
        }
      }
    }
    add_gram<NB>(hi, lo, acc);
  }
  store_gram<SP>(acc, lds, p.gram_to + id * SP * SP, wave, lane);
}

template <int SP>
__global__ __launch_bounds__(kThreads) void small_step_kernel(SmallArgs p, int64_t base) {
  constexpr int NB = SP / 16, KS = SP / 32, kBlocks = NB * (NB + 1) / 2, kPitch = SP + 8;
  constexpr int kMat = SP * kPitch * 2;   // bytes of one 16-bit matrix
  constexpr int kSums = (kWaves - 1) * kBlocks * 64 * 16;
  __shared__ __attribute__((aligned(16))) unsigned char lds[4 * kMat > kSums ? 4 * kMat : kSums];
  half_t* mat[4];   // A hi, A lo, C hi, C lo
#pragma unroll
  for (int q = 0; q < 4; ++q) mat[q] = reinterpret_cast<half_t*>(lds + q * kMat);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int64_t id = base + blockIdx.x, l = id / p.slabs;
  const int slab = (int)(id % p.slabs);
  const StartArgs& st = p.st;

  // (a vector load, ahead of the parts': a scalar one would be waited for on its own,
  // 0.5 us a step)
  int64_t at_own = 4 * l;
  asm volatile("" : "+v"(at_own));
  const f4 own = *(const f4*)(p.growth.coef + at_own);

  // A, from the slabs' parts in order
  constexpr int kQuads = SP * SP / 4 / kThreads;
  static_assert(kQuads * kThreads * 4 == SP * SP, "a quad a thread");
  f4 sum[kQuads];
#pragma unroll
  for (int q = 0; q < kQuads; ++q) sum[q] = f4{0.f, 0.f, 0.f, 0.f};
  const f4* parts = reinterpret_cast<const f4*>(p.gram + l * p.slabs * SP * SP);
#pragma unroll 4
  for (int i = 0; i < p.slabs; ++i)
#pragma unroll
    for (int q = 0; q < kQuads; ++q)
      sum[q] += parts[i * (SP * SP / 4) + q * kThreads + threadIdx.x];
#pragma unroll
  for (int q = 0; q < kQuads; ++q) {
    const int e = 4 * (q * kThreads + threadIdx.x);
    h4 hi, lo;
    split4(sum[q] * ldexpf(1.f, kScaleA - 2 * kScaleX), hi, lo);
    *(h4*)(mat[0] + e / SP * kPitch + e % SP) = hi;
    *(h4*)(mat[1] + e / SP * kPitch + e % SP) = lo;
  }
  float alpha = p.alpha, beta = p.beta, gamma = p.gamma;
  const float values[4] = {own[0], own[1], own[2], own[3]};
  float fc, fb, fa;
  hgemm::growth_factors(p.growth, values, fc, fb, fa);
  alpha *= fc;
  beta *= fb;
  gamma *= fa;
  auto frag = [&](int which, int block, int k) __attribute__((always_inline)) {
    return *(const h8*)(mat[which] + (16 * block + r) * kPitch + 32 * k + 8 * g);
  };
  __syncthreads();
  // C, block by block
  for (int q = wave; q < NB * NB; q += kWaves) {
    const int i = q / NB, j = q % NB;
    f4 c = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const h8 ah = frag(0, i, k), al = frag(1, i, k), bh = frag(0, j, k), bl = frag(1, j, k);
      c = mul(ah, bh, c);
      c = mul(ah, bl, c);
      c = mul(al, bh, c);
    }
    // rows 16 i + 4 g + v, column 16 j + r; stored as the other half, C being
    // symmetric: four values in a row
    f4 v;
    h4 hi, lo;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = 16 * i + 4 * g + e, at = row * kPitch + 16 * j + r;
      v[e] = alpha * c[e] + beta * ((float)mat[0][at] + (float)mat[1][at]) +
             (row == 16 * j + r ? gamma : 0.f);
    }
    split4(v, hi, lo);
    const int at = (16 * j + r) * kPitch + 16 * i + 4 * g;
    *(h4*)(mat[2] + at) = hi;
    *(h4*)(mat[3] + at) = lo;
  }
  __syncthreads();

  h8 ch[NB][KS], cl[NB][KS];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      ch[i][k] = frag(2, i, k);
      cl[i][k] = frag(3, i, k);
    }
  f4 acc[kBlocks];
#pragma unroll
  for (int q = 0; q < kBlocks; ++q) acc[q] = f4{0.f, 0.f, 0.f, 0.f};
  const bool tall = st.m > st.n;
  const int s = tall ? st.n : st.m, t = tall ? st.m : st.n;
  const int64_t columns = (int64_t)p.slabs * p.slab;
  const int out_size = p.out.type == kF32 ? 4 : 2;
  char* out = static_cast<char*>(p.out.O) + l * p.out.stride_o * out_size;
  // four values of the result in a row: row `row`, columns from `col` (of the
  // output as it lies)
  auto put = [&](int64_t row, int col, int cols, f4 v) __attribute__((always_inline)) {
    const int64_t at = row * p.out.ldo + col;
    if (p.out.type == kF32) {
      float* d = reinterpret_cast<float*>(out) + at;
      if (col + 4 <= cols) {
        __builtin_memcpy(d, &v, 16);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col + e < cols) d[e] = v[e];
      }
    } else {
      h4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[e] = p.out.type == GEMM_TYPE_BF16 ? f32_to_word<kFmtBF16>(v[e]) : f32_to_word<kFmtF16>(v[e]);
      half_t* d = reinterpret_cast<half_t*>(out) + at;
      if (col + 4 <= cols) {
        __builtin_memcpy(d, &o, 8);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col + e < cols) d[e] = o[e];
      }
    }
  };
  const float down = ldexpf(1.f, -kScaleA);
  const float end = ldexpf(1.f, -kScaleA - kScaleX) *
                    (p.last ? hgemm::growth_rate(values, p.growth.next, p.growth.next_most) : 1.f);
  for (int c = wave * kCols; c < p.slab; c += kWaves * kCols) {
    const int n0 = slab * p.slab + c;
    h8 xh[2][KS], xl[2][KS];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int64_t at = (l * columns + n0 + 16 * b + r) * SP + 32 * k + 8 * g;
        xh[b][k] = *(const h8*)(p.from[0] + at);
        xl[b][k] = *(const h8*)(p.from[1] + at);
      }
    h8 hi[NB], lo[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        f4 v = f4{0.f, 0.f, 0.f, 0.f}, w = v;
        if (!p.last || !tall) {
          // rows n0 + 16 b + 4 g + e of X^T C, column 16 i + r
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            v = mul(xh[b][k], ch[i][k], v);
            v = mul(xh[b][k], cl[i][k], v);
            v = mul(xl[b][k], ch[i][k], v);
          }
        }
        if (!p.last || tall) {
          // rows 16 i + 4 g + e of C X, column n0 + 16 b + r
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            w = mul(ch[i][k], xh[b][k], w);
            w = mul(cl[i][k], xh[b][k], w);
            w = mul(ch[i][k], xl[b][k], w);
          }
        }
        if (!p.last) {
          h4 h, u;
          split4(v * down, h, u);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            hi[i][4 * b + e] = h[e];
            lo[i][4 * b + e] = u[e];
          }
          split4(w * down, h, u);
          const int64_t at = (l * columns + n0 + 16 * b + r) * SP + 16 * i + 4 * g;
          *(h4*)(p.to[0] + at) = h;
          *(h4*)(p.to[1] + at) = u;
        } else if (!tall) {
          if (16 * i + r < s && n0 + 16 * b + 4 * g < t)
            put(16 * i + r, n0 + 16 * b + 4 * g, t, v * end);
        } else {
          if (n0 + 16 * b + r < t && 16 * i + 4 * g < s)
            put(n0 + 16 * b + r, 16 * i + 4 * g, s, w * end);
        }
      }
    if (!p.last) add_gram<NB>(hi, lo, acc);
  }
  if (!p.last)
    store_gram<SP>(acc, reinterpret_cast<f4*>(lds), p.gram_to + id * SP * SP, wave, lane);
}

}  // namespace

SmallPlan plan_small(int L, int s, int t) {
  SmallPlan p;
  p.side = s <= 32 ? 32 : 64;
  // slabs of whole turns of the waves; enough for the chip, few enough to add up
  constexpr int kTurn = kWaves * kCols;
  p.slabs = std::min(kMaxSlabs, (t + kTurn - 1) / kTurn);
  p.slab = (int)round_up((t + p.slabs - 1) / p.slabs, kCols);
  p.slabs = (t + p.slab - 1) / p.slab;
  p.x = round256((size_t)L * p.slabs * p.slab * p.side * 2);
  p.gram = round256((size_t)L * p.slabs * p.side * p.side * sizeof(float));
  return p;
}

hipError_t launch_small(const StartArgs& st, const SmallPlan& p, int steps, const float* coeffs,
                        const SmallOut& out, char* ws, hipStream_t stream) {
  half_t* x[2][2];
  float* gram[2];
  for (int i = 0; i < 2; ++i) {
    for (int v = 0; v < 2; ++v) x[i][v] = reinterpret_cast<half_t*>(ws + (2 * i + v) * p.x);
    gram[i] = reinterpret_cast<float*>(ws + 4 * p.x + i * p.gram);
  }
  SmallArgs a{};
  a.st = st;
  a.slabs = p.slabs;
  a.slab = p.slab;
  a.out = out;
  const int64_t wgs = (int64_t)st.L * p.slabs;
  a.to[0] = x[0][0];
  a.to[1] = x[0][1];
  a.gram_to = gram[0];
  hipError_t e = launch_tiles(p.side == 32 ? (const void*)small_start_kernel<32>
                                           : (const void*)small_start_kernel<64>,
                              a, wgs, kThreads, 0, stream);
  for (int k = 0; k < steps && e == hipSuccess; ++k) {
    const int i = k & 1;
    for (int v = 0; v < 2; ++v) {
      a.from[v] = x[i][v];
      a.to[v] = x[1 - i][v];
    }
    a.gram = gram[i];
    a.gram_to = gram[1 - i];
    a.alpha = ldexpf(coeffs[3 * k + 2], -kScaleA);
    a.beta = coeffs[3 * k + 1];
    a.gamma = ldexpf(coeffs[3 * k], kScaleA);
    a.growth = growth_of(st.coef, coeffs, k, steps);
    a.last = k + 1 == steps;
    e = launch_tiles(p.side == 32 ? (const void*)small_step_kernel<32>
                                  : (const void*)small_step_kernel<64>,
                     a, wgs, kThreads, 0, stream);
  }
  return e;
}

}  // namespace ortho
}  // namespace tune
}  // namespace mi355gemm

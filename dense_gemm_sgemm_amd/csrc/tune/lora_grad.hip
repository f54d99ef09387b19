// The gradients of low-rank adapters (tune.hpp says how rows are listed).
//
// A product of a few ranks by all columns, summed over an adapter's rows: bound
// by reading X and dC once.  Both operands have the summed index as their rows,
// while a matrix-core fragment wants eight of it in a lane.  `left` is small and
// is laid out so beforehand (pack_kernel); `right` is turned in registers: a
// lane loads 8 rows x 8 columns in 16-byte pieces and exchanges them, so that
// its eight fragments are eight neighbouring columns.  LDS is for adding up the
// waves alone (24 KB); any alignment.
// bf16, 4096 rows of X and of dC, 4096 columns each, one adapter of 16 ranks: 17 us
// (3.9 TB/s), and 19 in the three small launches (lists, packing, sums).
//
// A workgroup takes 128 columns, up to 32 ranks and a chunk of the steps, which
// its waves share; the waves' sums are added through LDS at the end of each
// adapter's steps in the chunk.  An adapter that lies in one chunk is stored at
// once, the others' chunks leave fp32 sums that a second kernel adds in order.
#include "tune.hpp"

namespace mi355gemm {
namespace tune {
namespace {

using hgemm::f4;
using hgemm::h8;
using hgemm::mfma16;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256, kWaves = kThreads / 64, kCols = 128;

constexpr int kListThreads = 1024, kListWaves = kListThreads / 64;

// Sum over the threads of a workgroup of kListThreads.
__device__ __forceinline__ int sum_all(int v, int* lds) {
#pragma unroll
  for (int k = 32; k >= 1; k /= 2) v += __shfl_xor(v, k);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < kListWaves; ++w) v += lds[w];
  return v;
}

// More adapters than kHistogram: one workgroup counts their rows in p.first (whole
// numbers: in any order) and adds up the steps.  An adapter's count goes where its
// rows will be listed.
__global__ __launch_bounds__(kListThreads) void count_kernel(GroupArgs p, int64_t) {
  __shared__ int lds[kListWaves];
  for (int i = threadIdx.x; i < p.S; i += kListThreads) p.first[i] = 0;
  __threadfence();
  __syncthreads();
  for (int m = threadIdx.x; m < p.M; m += kListThreads) {
    const long long id = p.ids[m];
    if (id >= 0 && id < p.S) atomicAdd(p.first + id, 1);
  }
  __threadfence();
  __syncthreads();
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  int before = 0;
  for (int a0 = 0; a0 < p.S; a0 += kListThreads) {
    const int a = a0 + threadIdx.x;
    // (from where the atomics left it)
    const int count = a < p.S ? __hip_atomic_load(p.first + a, __ATOMIC_RELAXED,
                                                  __HIP_MEMORY_SCOPE_AGENT) : 0;
    const int n = (count + 31) / 32;
    int sum = n;
#pragma unroll
    for (int k = 1; k < 64; k *= 2) {
      const int v = __shfl_up(sum, k);
      if (lane >= k) sum += v;
    }
    __syncthreads();
    if (lane == 63) lds[wave] = sum;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < kListWaves; ++w) {
      sum += w < wave ? lds[w] : 0;
      all += lds[w];
    }
    if (a < p.S) p.first[a] = before + sum - n;
    if (count) p.rows[32 * (int64_t)(before + sum - n)] = count;
    before += all;
  }
  if (threadIdx.x == 0) p.first[p.S] = before;
}

// Workgroup a lists the rows of adapter a, behind those of the adapters before
// it; workgroup S marks the steps that are left over.  Up to kHistogram adapters
// each workgroup counts all of them for itself (whole numbers: in any order).
// The workgroups past S turn the factors' stacks (below), which needs none of it.
struct ListJobs {
  GroupArgs g;
  int groups;   // workgroups of the lists, or 0
  TurnArgs turn[2];
  int64_t turns0;   // workgroups of the first
};
__device__ void list_rows(const GroupArgs& p, int a, int* lds, int* bins) {
  int before = 0, count = 0;   // before: steps
  if (p.S <= kHistogram) {
    for (int i = threadIdx.x; i < p.S; i += kListThreads) bins[i] = 0;
    __syncthreads();
    for (int m = threadIdx.x; m < p.M; m += kListThreads) {
      const long long id = p.ids[m];
      if (id >= 0 && id < p.S) atomicAdd(bins + (int)id, 1);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a; i += kListThreads) before += (bins[i] + 31) / 32;
    if (a < p.S) count = bins[a];
    before = sum_all(before, lds);
    if (threadIdx.x == 0) p.first[a] = before;
  } else {
    before = p.first[a];
    if (a < p.S && p.first[a + 1] != before) count = p.rows[32 * (int64_t)before];
    __syncthreads();   // (its place is written below)
  }
  if (a == p.S) {
    for (int i = before + threadIdx.x; i < p.steps; i += kListThreads) p.step_adapter[i] = -1;
    return;
  }
  const int steps = (count + 31) / 32;
  for (int i = threadIdx.x; i < steps; i += kListThreads) p.step_adapter[before + i] = a;
  int* rows = p.rows + 32 * (int64_t)before;
  for (int i = count + threadIdx.x; i < 32 * steps; i += kListThreads) rows[i] = -1;
  int at = 0;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int64_t m0 = 0; m0 < p.M && at < count; m0 += kListThreads) {
    const int64_t m = m0 + threadIdx.x;
    const bool mine = m < p.M && p.ids[m] == a;
    const uint64_t votes = __ballot(mine);
    __syncthreads();
    if (lane == 0) lds[wave] = __popcll(votes);
    __syncthreads();
    int pos = at;
#pragma unroll
    for (int w = 0; w < kListWaves; ++w) {
      pos += w < wave ? lds[w] : 0;
      at += lds[w];
    }
    if (mine) rows[pos + __popcll(votes & ((uint64_t(1) << lane) - 1))] = (int)m;
  }
}

// A thread 8 inner values of one outer index; neighbouring threads neighbouring
// outer indices.
__device__ __forceinline__ void turn(const TurnArgs& p, int64_t id) {
  int64_t t = id * kListThreads + threadIdx.x;
  const int o = (int)(t % p.outer);
  t /= p.outer;
  const int i = (int)(t % (p.inner_p / 8)) * 8;
  const int64_t l = t / (p.inner_p / 8);
  if (l >= p.count) return;
  const half_t* src = p.src + l * p.stride_s + (int64_t)i * p.lds + o;
  h8 v = {};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (i + e < p.inner) v[e] = src[e * p.lds];
  *(h8*)(p.dst + l * p.stride_d + (int64_t)o * p.ldd + i) = v;
}

__global__ __launch_bounds__(kListThreads) void list_kernel(ListJobs p, int64_t base) {
  __shared__ int lds[kListWaves], bins[kHistogram];
  int64_t id = base + blockIdx.x;
  if (id < p.groups) {
    list_rows(p.g, (int)id, lds, bins);
    return;
  }
  id -= p.groups;
  const bool second = id >= p.turns0;
  turn(second ? p.turn[1] : p.turn[0], second ? id - p.turns0 : id);
}

// A step's 32 rows of `left`, ranks as rows, in two 16-bit values times a power
// of two that brings the largest to 2^13 .. 2^14 (tune.hpp); step_factor undoes
// it and has the adapter's scale.
template <int FMT>
__global__ __launch_bounds__(kThreads) void pack_kernel(GradArgs p, int64_t base) {
  __shared__ int row[32];
  __shared__ float part[kWaves];
  const int64_t id = base + blockIdx.x;
  const GradJob& job = p.job[id / p.g.steps];
  if (job.out == nullptr) return;
  const int step = (int)(id % p.g.steps);
  const int a = p.g.step_adapter[step];
  if (a < 0) return;
  if (threadIdx.x < 32) row[threadIdx.x] = p.g.rows[32 * (int64_t)step + threadIdx.x];
  __syncthreads();
  float top = 0.f;
  for (int t = threadIdx.x; t < 32 * p.R; t += kThreads) {
    const int m = row[t / p.R];
    if (m < 0) continue;
    const float v = fabsf(job.left[m * job.ld_left + t % p.R]);
    top = fmaxf(top, v < __builtin_inff() ? v : 0.f);
  }
#pragma unroll
  for (int k = 32; k >= 1; k /= 2) top = fmaxf(top, __shfl_xor(top, k));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
  __syncthreads();
  top = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
  float up, down;
  scale_for(top, up, down);
  if (threadIdx.x == 0) job.step_factor[step] = down * (p.scales ? p.scales[a] : 1.f);
  const int64_t ld = 32 * (int64_t)p.g.steps, half = ld * p.padded;
  // a thread a rank and 8 rows
  for (int t = threadIdx.x; t < 4 * p.padded; t += kThreads) {
    const int rank = t >> 2, q = t & 3;
    h8 hi = {}, lo = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int m = row[8 * q + i];
      if (m < 0 || rank >= p.R) continue;
      half_t a, b;
      split_value<FMT>(job.left[m * job.ld_left + rank] * up, a, b);
      hi[i] = a;
      lo[i] = b;
    }
    half_t* dst = job.pack + rank * ld + 32 * (int64_t)step + 8 * q;
    *(h8*)dst = hi;
    *(h8*)(dst + half) = lo;
  }
}

// Where a workgroup's sums of an adapter go: 16 RB ranks x 128 columns, lane
// (g, j) holding ranks 16 q + 4 g + v, columns c0 + 8 j + e.
template <int FMT, int RB>
__device__ __forceinline__ void store_out(const GradArgs& p, const GradJob& job, int a, int first,
                                          int c0, int lane, const f4 (&acc)[RB][8]) {
  const int g = lane >> 4, col = c0 + 8 * (lane & 15);
  half_t* out = job.out + a * job.stride_o;
#pragma unroll
  for (int q = 0; q < RB; ++q) {
    const int rank = first + 16 * q + 4 * g;
    if (!job.transposed) {
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        if (rank + v >= p.R || col >= job.cols) continue;
        half_t* dst = out + (int64_t)(rank + v) * job.ldo + col;
        h8 o;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = f32_to_word<FMT>(acc[q][e][v]);
        if (col + 8 <= job.cols) {
          __builtin_memcpy(dst, &o, 16);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (col + e < job.cols) dst[e] = o[e];
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (col + e >= job.cols || rank >= p.R) continue;
        half_t* dst = out + (int64_t)(col + e) * job.ldo + rank;
        hgemm::h4 o;
#pragma unroll
        for (int v = 0; v < 4; ++v) o[v] = f32_to_word<FMT>(acc[q][e][v]);
        if (rank + 4 <= p.R) {
          __builtin_memcpy(dst, &o, 8);
        } else {
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (rank + v < p.R) dst[v] = o[v];
        }
      }
    }
  }
}

// Partial sums: the f4 of (slot, block of columns, group of ranks), [q][e][lane].
// A chunk leaves two at most, of an adapter that goes on from the chunk before
// and of one that begins in it and goes on to the next: slots 2 chunk and 2 chunk
// + 1.  With fewer adapters than chunks it is slot chunk + a: no two share one,
// since each next place in the order of the steps has a later chunk or adapter.
__device__ __forceinline__ int partial_slot(const GradArgs& p, int chunk, int a, bool begins) {
  return p.by_adapter ? chunk + a : 2 * chunk + begins;
}
__device__ __forceinline__ f4* partial_at(const GradArgs& p, const GradJob& job, int slot,
                                          int block, int group, int rb) {
  return reinterpret_cast<f4*>(job.partial) +
         (((int64_t)slot * job.blocks + block) * p.groups + group) * (rb * 8 * 64);
}

template <int FMT, int RB>
__global__ __launch_bounds__(kThreads) void grad_kernel(GradArgs p, int64_t base) {
  __shared__ f4 lds[(kWaves - 1) * 8 * 64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, j = lane & 15;
  int64_t id = base + blockIdx.x;
  const int blocks0 = p.job[0].blocks, blocks = blocks0 + p.job[1].blocks;
  int block = (int)(id % blocks);
  id /= blocks;
  const int group = (int)(id % p.groups);
  const int chunk = (int)(id / p.groups);
  const int which = block >= blocks0;
  if (which) block -= blocks0;
  const GradJob& job = p.job[which];
  const int first = group * 16 * RB, c0 = block * kCols, col = c0 + 8 * j;
  const int s0 = chunk * p.chunk_steps;
  const int s1 = s0 + p.chunk_steps < p.g.steps ? s0 + p.chunk_steps : p.g.steps;
  const int64_t ld = 32 * (int64_t)p.g.steps, half = ld * p.padded;
  const half_t* pack[RB];
#pragma unroll
  for (int q = 0; q < RB; ++q) {
    // (ranks past the padded ones repeat the last, unstored)
    const int rank = first + 16 * q + j;
    pack[q] = job.pack + (rank < p.padded ? rank : p.padded - 1) * ld + 8 * g;
  }
  int s = s0;
  while (s < s1) {
    const int a = p.g.step_adapter[s];
    if (a < 0) break;
    int end = s + 1;   // the adapter's last step in the chunk
    while (end < s1 && p.g.step_adapter[end] == a) ++end;
    f4 acc[RB][8];
#pragma unroll
    for (int q = 0; q < RB; ++q)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[q][e] = f4{0.f, 0.f, 0.f, 0.f};
    for (int t = s + wave; t < end; t += kWaves) {
      const int* rows = p.g.rows + 32 * (int64_t)t + 8 * g;
      const i4 ra = *(const i4*)rows, rb = *(const i4*)(rows + 4);
      h8 x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int m = i < 4 ? ra[i & 3] : rb[i & 3];
        x[i] = h8{};
        if (m >= 0 && col < job.cols) {
          const half_t* src = job.right + (int64_t)m * job.ld_right + col;
          if (col + 8 <= job.cols) {
            __builtin_memcpy(&x[i], src, 16);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (col + e < job.cols) x[i][e] = src[e];
          }
        }
      }
      h8 hi[RB], lo[RB];
#pragma unroll
      for (int q = 0; q < RB; ++q) {
        hi[q] = *(const h8*)(pack[q] + 32 * (int64_t)t);
        lo[q] = *(const h8*)(pack[q] + half + 32 * (int64_t)t);
      }
      const float f = job.step_factor[t];
      turn8(x);
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int q = 0; q < RB; ++q) {
          f4 d = mfma16<FMT>(hi[q], x[e], f4{0.f, 0.f, 0.f, 0.f});
          d = mfma16<FMT>(lo[q], x[e], d);
          acc[q][e] += d * f;
          asm volatile("" : "+v"(acc[q][e]));   // (each at once: registers)
        }
    }
    add_up<RB>(acc, lds, wave, lane);
    if (wave == 0) {
      const bool begins = s == 0 || p.g.step_adapter[s - 1] != a;
      const bool whole = begins && (end == p.g.steps || p.g.step_adapter[end] != a);
      if (whole) {
        store_out<FMT, RB>(p, job, a, first, c0, lane, acc);
      } else {
        f4* dst = partial_at(p, job, partial_slot(p, chunk, a, begins), block, group, RB);
#pragma unroll
        for (int q = 0; q < RB; ++q)
#pragma unroll
          for (int e = 0; e < 8; ++e) dst[(q * 8 + e) * 64 + lane] = acc[q][e];
      }
    }
    s = end;
  }
}

// The adapters that lie in several chunks, and those without rows (zeros): a
// workgroup for 128 columns and 16 RB ranks, its waves every so many of the chunks.
template <int FMT, int RB>
__global__ __launch_bounds__(kThreads) void join_kernel(GradArgs p, int64_t base) {
  __shared__ f4 lds[(kWaves - 1) * 8 * 64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t id = base + blockIdx.x;
  const int blocks0 = p.job[0].blocks, blocks = blocks0 + p.job[1].blocks;
  const int group = (int)(id % p.groups);
  id /= p.groups;
  int block = (int)(id % blocks);
  const int a = (int)(id / blocks);
  const int which = block >= blocks0;
  if (which) block -= blocks0;
  const GradJob& job = p.job[which];
  const int before = p.g.first[a], steps = p.g.first[a + 1] - before;
  const int from = before / p.chunk_steps;
  const int to = steps ? (before + steps - 1) / p.chunk_steps : from;
  if (steps && from == to) return;   // stored already
  f4 acc[RB][8];
#pragma unroll
  for (int q = 0; q < RB; ++q)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[q][e] = f4{0.f, 0.f, 0.f, 0.f};
  if (steps)
    for (int c = from + wave; c <= to; c += kWaves) {
      const f4* src = partial_at(p, job, partial_slot(p, c, a, c == from), block, group, RB);
      f4 v[RB][8];
#pragma unroll
      for (int q = 0; q < RB; ++q)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[q][e] = src[(q * 8 + e) * 64 + lane];
      __builtin_amdgcn_sched_barrier(0);   // (all loads, then the sums)
#pragma unroll
      for (int q = 0; q < RB; ++q)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[q][e] += v[q][e];
    }
  add_up<RB>(acc, lds, wave, lane);
  if (wave > 0) return;
  store_out<FMT, RB>(p, job, a, group * 16 * RB, block * kCols, lane, acc);
}

__global__ __launch_bounds__(kThreads) void widen_kernel(WidenArgs p, int64_t base) {
  int64_t t = (base + blockIdx.x) * kThreads + threadIdx.x;
  const int c = (int)(t % (p.cols_p / 8)) * 8;
  t /= p.cols_p / 8;
  const int64_t l = t / p.rows;
  if (l >= p.count) return;
  const half_t* src = p.src + l * p.stride_s + (t - l * p.rows) * p.lds;
  h8 v = {};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c + e < p.cols) v[e] = src[c + e];
  *(h8*)(p.dst + t * p.cols_p + c) = v;
}
__global__ __launch_bounds__(kThreads) void tail_kernel(TailArgs p, int64_t base) {
  const int64_t t = (base + blockIdx.x) * kThreads + threadIdx.x;
  const int64_t row = t / 8;
  const int c = (int)(t % 8) * 8;
  if (row >= p.rows_p) return;
  h8 v = {};
  if (row < p.rows) {
    const half_t* src = p.src + row * p.lds + p.K - 64 + c;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e >= 64 - p.K % 64) v[e] = src[e];
  }
  *(h8*)(p.dst + row * 64 + c) = v;
}
int64_t turn_blocks(const TurnArgs& p) {
  return ((int64_t)p.outer * (p.inner_p / 8) * p.count + kListThreads - 1) / kListThreads;
}

template <int FMT, int RB>
hipError_t launch_rb(const GradArgs& p, hipStream_t stream) {
  const int64_t blocks = (int64_t)p.job[0].blocks + p.job[1].blocks;
  hipError_t e = launch_tiles((const void*)grad_kernel<FMT, RB>, p, blocks * p.groups * p.chunks,
                              kThreads, 0, stream);
  if (e != hipSuccess) return e;
  return launch_tiles((const void*)join_kernel<FMT, RB>, p, blocks * p.groups * p.g.S, kThreads, 0,
                      stream);
}

}  // namespace

hipError_t launch_lists(const GroupArgs* group, const TurnArgs* turns, int count,
                        hipStream_t stream) {
  ListJobs jobs{};
  int64_t blocks = 0;
  if (group) {
    jobs.g = *group;
    jobs.groups = group->S + 1;
    if (group->S > kHistogram) {
      const hipError_t e =
          launch_tiles((const void*)count_kernel, *group, 1, kListThreads, 0, stream);
      if (e != hipSuccess) return e;
    }
  }
  for (int i = 0; i < count; ++i) {
    jobs.turn[i] = turns[i];
    if (i == 0) jobs.turns0 = turn_blocks(turns[i]);
    blocks += turn_blocks(turns[i]);
  }
  return launch_tiles((const void*)list_kernel, jobs, jobs.groups + blocks, kListThreads, 0, stream);
}

// Chunks so that some 1024 workgroups share the work (adapters of few rows are a
// step each: a chunk of several would take them one after another).
GradPlan plan_grad(int M, int N, int K, int R, int S) {
  GradPlan p;
  p.steps = max_steps(M, S);
  p.padded = (int)round_up(R, 16);
  p.rb = R <= 16 ? 1 : 2;
  p.groups = (R + 16 * p.rb - 1) / (16 * p.rb);
  const int64_t cols[2] = {K, N};
  const int64_t blocks = ((cols[0] + kCols - 1) / kCols + (cols[1] + kCols - 1) / kCols) * p.groups;
  const int64_t want = std::max<int64_t>(1, 1024 / std::max<int64_t>(1, blocks));
  p.chunk_steps = std::max<int>(1, (int)((p.steps + want - 1) / want));
  p.chunks = (p.steps + p.chunk_steps - 1) / p.chunk_steps;
  p.by_adapter = S < p.chunks;
  p.pack = round256((size_t)2 * p.padded * p.steps * 64);
  for (int i = 0; i < 2; ++i)
    p.partial[i] = (size_t)(p.by_adapter ? p.chunks + S : 2 * p.chunks) *
                   ((cols[i] + kCols - 1) / kCols) * p.groups * p.rb * 8 * 64 * sizeof(f4);
  return p;
}

hipError_t launch_adapter_grads(int fmt, const GradArgs& p, const GradPlan& plan,
                                hipStream_t stream) {
  const hipError_t e = launch_tiles(fmt == kFmtBF16 ? (const void*)pack_kernel<kFmtBF16>
                                                    : (const void*)pack_kernel<kFmtF16>,
                                    p, 2 * (int64_t)p.g.steps, kThreads, 0, stream);
  if (e != hipSuccess) return e;
  if (fmt == kFmtBF16)
    return plan.rb == 1 ? launch_rb<kFmtBF16, 1>(p, stream) : launch_rb<kFmtBF16, 2>(p, stream);
  return plan.rb == 1 ? launch_rb<kFmtF16, 1>(p, stream) : launch_rb<kFmtF16, 2>(p, stream);
}

hipError_t launch_tail(const TailArgs& p, hipStream_t stream) {
  return launch_tiles((const void*)tail_kernel, p, ((int64_t)p.rows_p * 8 + kThreads - 1) / kThreads,
                      kThreads, 0, stream);
}

hipError_t launch_widen(const WidenArgs& p, hipStream_t stream) {
  const int64_t threads = (int64_t)p.count * p.rows * (p.cols_p / 8);
  return launch_tiles((const void*)widen_kernel, p, (threads + kThreads - 1) / kThreads, kThreads,
                      0, stream);
}

}  // namespace tune
}  // namespace mi355gemm

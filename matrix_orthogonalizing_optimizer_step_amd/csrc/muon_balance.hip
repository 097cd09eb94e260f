// The balance loss of a mixture's router, with the experts' token counts and the
// gradient for the logits.  With p_t the softmax (or the sigmoids over their sum) of
// token t's logits z_t and f_e = E count_e / (K T) fixed by the choices made,
//   L = alpha / S sum_s sum_e f_e mean_t p_te = alpha / S sum_s 1 / T_s sum_t <f, p_t>
//   dL/dz_te = alpha / (S T_s) slope_te (f_e - <f, p_t>),
// slope = p (softmax) or s (1 - s) / sum s (sigmoids s).  So once the counts are
// there one pass over the logits gives both: a row's <f, p> is its share of the loss
// and what its gradient needs; no mean of p is kept.  Since the p of a row add up to
// 1, d = f - min f stands in for f, made from the difference of the counts: near
// balance, where f_e - <f, p> is a small difference, less is lost, and where all experts
// have as many tokens the gradient is 0.
//
// Two launches: the choices are counted in LDS, a partial count for each block; then
// every block adds the partial counts of its sequence up to f, takes its rows, and
// the last block to finish adds the blocks' sums in their order, so results do not
// depend on timing.  Small calls do all of it in one block and one launch (5.5 us).
// 32768 x 256 bf16 with the gradient: counts 4 us, rows 18 to 20.  Those issue 39 vector
// instructions an element (counted; with the counts' sums and the reductions over a row),
// which alone would take 8.6 us, the logits' and the gradient's way through memory 5.
// 16 x 2049 x 61 fp32 sigmoid, padded to 64: 86 an element, 4.8 us, of 12.  The rest is
// waiting: four waves a SIMD, the reductions' chains, the last block's sum.
//
// The blocks' sums are all that passes from block to block within a launch.  They go
// by agent-scope atomic stores, which write through to memory, and are waited for
// before the block is counted as done; a release of everything the block wrote would
// write back the XCD's whole L2 for each of a thousand blocks.
#include "../../include/muon.h"
#include "muon_convert.h"
#include "muon_internal.h"

namespace muon {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef u32x4_t u32x4_a2 __attribute__((aligned(2)));
typedef u32x4_t u32x4_a4 __attribute__((aligned(4)));

constexpr int kMaxExperts = MUON_MAX_EXPERTS;
constexpr int kThreads = 1024;      // of a block, 512 for rows of more than 512 experts (registers)
constexpr int kSmallThreads = 256;  // where one block does everything
constexpr int kCountThreads = 1024;
constexpr int kElems = 8;  // of a row, consecutive, in a lane

struct BalanceArgs {
  int sequences, tokens, experts, top;
  const void* logits;
  int64_t stride;          // of rows of the logits, in elements
  const void* index;       // rows x top
  int wide;                // 64-bit indices
  const uint8_t* mask;     // or null
  int sigmoid;
  float coefficient;       // alpha / S
  const float* grad_scale;
  float* loss;
  int32_t* counts;
  void* grad;              // or null
  int accumulate;
  int count_blocks, blocks;  // of a sequence; count_blocks 0: one block does everything
  // workspace: partial counts [sequence][count block][experts + 1], the last one that
  // of the tokens; sums [sequence][block]; how many blocks are done
  int32_t* partial;
  double* sums;
  int32_t* done;
};

__device__ __forceinline__ bool counted(const BalanceArgs& a, int64_t row) { return a.mask == nullptr || a.mask[row] != 0; }

// Choices and tokens of rows first .. last - 1 into bins (experts + 1 of them).
__device__ __forceinline__ void count_rows(const BalanceArgs& a, int64_t first, int64_t last, int32_t* bins) {
  const uint32_t end = static_cast<uint32_t>(last * a.top);  // under 2^31
  constexpr int kAhead = 8;  // loads under way
  for (uint32_t p0 = static_cast<uint32_t>(first * a.top) + threadIdx.x; p0 < end; p0 += kAhead * blockDim.x) {
    int64_t e[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const uint32_t p = p0 + k * blockDim.x;
      e[k] = p >= end ? -1 : a.wide ? static_cast<const int64_t*>(a.index)[p] : static_cast<const int32_t*>(a.index)[p];
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (e[k] >= 0 && e[k] < a.experts && counted(a, (p0 + k * blockDim.x) / static_cast<uint32_t>(a.top)))
        atomicAdd(bins + e[k], 1);
  }
  if (a.mask == nullptr) {
    if (threadIdx.x == 0) atomicAdd(bins + a.experts, static_cast<int32_t>(last - first));
  } else {
    int n = 0;
    for (int64_t r = first + threadIdx.x; r < last; r += blockDim.x) n += a.mask[r] != 0;
    if (n > 0) atomicAdd(bins + a.experts, n);
  }
}

__global__ __launch_bounds__(kCountThreads) void balance_count_kernel(BalanceArgs a) {
  __shared__ int32_t bins[kMaxExperts + 1];
  for (int e = threadIdx.x; e <= a.experts; e += kCountThreads) bins[e] = 0;
  __syncthreads();
  const int64_t base = static_cast<int64_t>(blockIdx.y) * a.tokens;
  const int64_t first = static_cast<int64_t>(a.tokens) * blockIdx.x / a.count_blocks;
  const int64_t last = static_cast<int64_t>(a.tokens) * (blockIdx.x + 1) / a.count_blocks;
  count_rows(a, base + first, base + last, bins);
  __syncthreads();
  int32_t* out = a.partial + (static_cast<int64_t>(blockIdx.y) * a.count_blocks + blockIdx.x) * (a.experts + 1);
  for (int e = threadIdx.x; e <= a.experts; e += kCountThreads) out[e] = bins[e];
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    for (int e = threadIdx.x; e < a.experts; e += kCountThreads) a.counts[e] = 0;
    if (threadIdx.x == 0) *a.done = 0;
  }
}

template <int CTRL, class T>
__device__ __forceinline__ T dpp(T x) {
  return __builtin_bit_cast(T, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;  // quads, reversal within 8 and 16 lanes

// Over L neighbouring lanes, the same result in each of them.
template <int L, class T, class F>
__device__ __forceinline__ T lanes(T x, F op) {
  if constexpr (L >= 2) x = op(x, dpp<kXor1>(x));
  if constexpr (L >= 4) x = op(x, dpp<kXor2>(x));
  if constexpr (L >= 8) x = op(x, dpp<kHalfMirror>(x));
  if constexpr (L >= 16) x = op(x, dpp<kMirror>(x));
  if constexpr (L >= 32) x = op(x, __shfl_xor(x, 16));
  if constexpr (L >= 64) x = op(x, __shfl_xor(x, 32));
  return x;
}
template <int L>
__device__ __forceinline__ float lanes_sum(float x) {
  return lanes<L>(x, [](float a, float b) { return a + b; });
}
template <int L>
__device__ __forceinline__ float lanes_max(float x) {
  return lanes<L>(x, [](float a, float b) { return fmaxf(a, b); });
}

// Elements c .. c + 7 of a row of n, `none` behind its end.
template <int D>
__device__ __forceinline__ void load8(const void* p, int64_t row, int c, int n, float none, float* x) {
  if (c + kElems <= n) {
    if constexpr (D == kF32) {
      const u32x4_t lo = *reinterpret_cast<const u32x4_a4*>(static_cast<const float*>(p) + row + c);
      const u32x4_t hi = *reinterpret_cast<const u32x4_a4*>(static_cast<const float*>(p) + row + c + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = __uint_as_float(lo[e]);
        x[4 + e] = __uint_as_float(hi[e]);
      }
    } else {
      const u32x4_t v = *reinterpret_cast<const u32x4_a2*>(static_cast<const uint16_t*>(p) + row + c);
#pragma unroll
      for (int e = 0; e < kElems; ++e) {
        const uint16_t h = static_cast<uint16_t>((e & 1) ? v[e >> 1] >> 16 : v[e >> 1]);
        x[e] = D == kBF16 ? bf16_to_f32(h) : f16_to_f32(h);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < kElems; ++e) x[e] = c + e < n ? load_as_f32(p, row + c + e, D) : none;
  }
}

template <int D>
__device__ __forceinline__ void store8(void* p, int64_t row, int c, int n, const float* x) {
  if (c + kElems <= n) {
    if constexpr (D == kF32) {
      float* q = static_cast<float*>(p) + row + c;
      *reinterpret_cast<u32x4_a4*>(q) = (u32x4_t){__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                                                  __float_as_uint(x[3])};
      *reinterpret_cast<u32x4_a4*>(q + 4) = (u32x4_t){__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]),
                                                      __float_as_uint(x[7])};
    } else {
      u32x4_t v;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = D == kBF16 ? f32x2_to_bf16x2(x[2 * e], x[2 * e + 1]) : f32x2_to_f16x2(x[2 * e], x[2 * e + 1]);
      *reinterpret_cast<u32x4_a2*>(static_cast<uint16_t*>(p) + row + c) = v;
    }
  } else {
#pragma unroll
    for (int e = 0; e < kElems; ++e)
      if (c + e < n) store_from_f32(p, row + c + e, D, x[e]);
  }
}

// e^x for x <= 0 (NaN for NaN), 0 under the normal range: 2^h (1 + l ln 2) with h + l = x
// log2(e), l what the rounding of h left, so that the result is good to two steps for
// every x; half the instructions of the general function.
__device__ __forceinline__ float exp_of(float x) {
  constexpr float kLog2e = 0x1.715476p+0f, kRest = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
  x = __builtin_elementwise_maximum(x, -128.0f);  // -infinity has no l
  const float h = x * kLog2e, l = fmaf(x, kRest, fmaf(x, kLog2e, -h));
  const float e = __builtin_amdgcn_exp2f(h);
  return fmaf(e, l * kLn2, e);
}

// Sigmoids that add up to less than this leave fp32's range, or are about to (2^-126 is
// nothing beside it): every logit is under -44, where 1 + e^z is 1 and p the softmax, each
// to 2^-64 of itself.
constexpr float kSmallSum = 0x1p-64f;

// The gradient's factor slope for a row's logits x (which are used up); returns <d, p>.
// some: whether any expert has p > 0.  small: the sigmoids are too small, nothing else is
// set (p is the softmax).
template <int L, int N>
__device__ __forceinline__ float row_scores(float (&x)[N], float (&slope)[N], const float (&d)[N], bool sigmoid, bool* some,
                                            bool* small) {
  float sum = 0.0f, inner = 0.0f;
  *small = false;
  if (sigmoid) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float t = exp_of(-fabsf(x[e])), q = 1.0f / (1.0f + t);  // the sigmoid of |z|
      x[e] = x[e] < 0.0f ? t * q : q;
      slope[e] = t * q * q;
      sum += x[e];
    }
    sum = lanes_sum<L>(sum);
    *some = true;
    *small = sum < kSmallSum;
    const float inverse = 1.0f / sum;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      slope[e] *= inverse;
      inner += d[e] * (x[e] * inverse);
    }
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int e = 0; e < N; ++e) m = fmaxf(m, x[e]);
    m = lanes_max<L>(m);
    m = m == -INFINITY ? 0.0f : m;  // nothing to choose from: p = 0
#pragma unroll
    for (int e = 0; e < N; ++e) {
      x[e] = exp_of(x[e] - m);
      sum += x[e];
    }
    sum = lanes_sum<L>(sum);
    *some = sum != 0.0f;
    const float inverse = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      slope[e] = x[e] * inverse;
      inner += d[e] * slope[e];
    }
  }
  return lanes_sum<L>(inner);
}

// Rows first, first + step, ... under last: their <f, p> added up (this thread's
// share of them), their gradients written.  L lanes take a row, lane `o` of them
// elements 8 (o + L v).  The next row's logits are on their way meanwhile.
template <int D, int L, int NV>
__device__ __forceinline__ void load_row(const BalanceArgs& a, int64_t r, float (&x)[NV * kElems]) {
#pragma unroll
  for (int v = 0; v < NV; ++v)
    load8<D>(a.logits, r * a.stride, kElems * (static_cast<int>(threadIdx.x) % L + L * v), a.experts, -INFINITY,
             x + v * kElems);
}

// (x: the thread's first row, valid: whether it counts)
template <int D, int L, int NV>
__device__ __forceinline__ float take_rows(const BalanceArgs& a, const int32_t* bins, int64_t first, int64_t last, int step,
                                           float scale, float (&x)[NV * kElems], bool valid) {
  constexpr int N = NV * kElems;
  const int o = threadIdx.x % L, E = a.experts, tokens = bins[E];
  const float unit = tokens > 0 ? static_cast<float>(E) / (static_cast<float>(a.top) * static_cast<float>(tokens)) : 0.0f;
  int least = INT32_MAX;  // count of an expert
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int e = 0; e < kElems; ++e) {
      const int c = kElems * (o + L * v) + e, n = c < E ? bins[c] : INT32_MAX;
      least = n < least ? n : least;
    }
  least = lanes<L>(least, [](int p, int q) { return p < q ? p : q; });
  const float all = static_cast<float>(least) * unit;  // of f, in every expert's
  float d[N];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int e = 0; e < kElems; ++e) {
      const int c = kElems * (o + L * v) + e;
      d[v * kElems + e] = c < E ? static_cast<float>(bins[c] - least) * unit : 0.0f;
    }
  const float by = tokens > 0 ? scale / static_cast<float>(tokens) : 0.0f;  // of the gradient
  float total = 0.0f;
  int64_t r = first + threadIdx.x / L;
  // all lanes of a row are in the loop together (they share a row)
  while (r < last) {
    const int64_t after = r + step;
    const bool valid_after = after < last && counted(a, after);
    float next[N], g[N];
    if (valid_after) load_row<D, L, NV>(a, after, next);
    if (valid) {
      bool some, small;
      float inner = row_scores<L>(x, g, d, a.sigmoid != 0, &some, &small);
      if (small) {  // the same in all lanes of a row
        load_row<D, L, NV>(a, r, x);
        inner = row_scores<L>(x, g, d, false, &some, &small);
      }
      if (o == 0) total += some ? all + inner : 0.0f;
#pragma unroll
      for (int e = 0; e < N; ++e) g[e] *= (d[e] - inner) * by;
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) g[e] = 0.0f;
    }
    if (a.grad != nullptr && (valid || !a.accumulate)) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = kElems * (o + L * v);
        if (c < E) {
          if (a.accumulate) {
            float was[kElems];
            load8<D>(a.grad, r * E, c, E, 0.0f, was);
#pragma unroll
            for (int e = 0; e < kElems; ++e) g[v * kElems + e] += was[e];
          }
          store8<D>(a.grad, r * E, c, E, g + v * kElems);
        }
      }
    }
    r = after;
    valid = valid_after;
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = next[e];
  }
  return total;
}

__device__ __forceinline__ double block_sum(double x, double* waves) {
#pragma unroll
  for (int m = 1; m < 64; m *= 2) x += __shfl_xor(x, m);
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = x;
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < static_cast<int>(blockDim.x) / 64; ++w) s += waves[w];
  __syncthreads();
  return s;
}

template <int D, int L, int NV>
__global__ __launch_bounds__(kThreads / NV) void balance_rows_kernel(BalanceArgs a) {
  __shared__ int32_t bins[kMaxExperts + 1];
  __shared__ double waves[kThreads / 64];
  __shared__ int last_block;
  const int E = a.experts;
  const float alpha = a.coefficient, scale = alpha * (a.grad_scale != nullptr ? *a.grad_scale : 1.0f);
  if (a.count_blocks == 0) {  // one block
    double total = 0.0;
    for (int e = threadIdx.x; e < E; e += blockDim.x) a.counts[e] = 0;
    for (int s = 0; s < a.sequences; ++s) {
      __syncthreads();
      for (int e = threadIdx.x; e <= E; e += blockDim.x) bins[e] = 0;
      __syncthreads();
      const int64_t base = static_cast<int64_t>(s) * a.tokens;
      count_rows(a, base, base + a.tokens, bins);
      __syncthreads();
      for (int e = threadIdx.x; e < E; e += blockDim.x) a.counts[e] += bins[e];
      const int64_t r = base + threadIdx.x / L;
      const bool valid = r < base + a.tokens && counted(a, r);
      float x[NV * kElems];
      if (valid) load_row<D, L, NV>(a, r, x);
      const float sum = take_rows<D, L, NV>(a, bins, base, base + a.tokens, blockDim.x / L, scale, x, valid);
      total += bins[E] > 0 ? static_cast<double>(sum) / bins[E] : 0.0;
    }
    total = block_sum(total, waves);
    if (threadIdx.x == 0) *a.loss = static_cast<float>(total * alpha);
    return;
  }
  const int s = blockIdx.y;
  const int64_t base = static_cast<int64_t>(s) * a.tokens;
  const int64_t first = base + static_cast<int64_t>(a.tokens) * blockIdx.x / a.blocks;
  const int64_t last = base + static_cast<int64_t>(a.tokens) * (blockIdx.x + 1) / a.blocks;
  const int64_t r = first + threadIdx.x / L;
  const bool valid = r < last && counted(a, r);
  float x[NV * kElems];
  if (valid) load_row<D, L, NV>(a, r, x);  // on its way while the counts are added up
  const int32_t* partial = a.partial + static_cast<int64_t>(s) * a.count_blocks * (E + 1);
  for (int e = threadIdx.x; e <= E; e += blockDim.x) bins[e] = 0;
  __syncthreads();
  // as many threads for a bin as there are, eight loads at a time under way
  const int per = static_cast<int>(blockDim.x) / (E + 1) > 0 ? static_cast<int>(blockDim.x) / (E + 1) : 1;
  for (int p = threadIdx.x; p < per * (E + 1); p += blockDim.x) {
    const int e = p % (E + 1);
    int n = 0;
    for (int b0 = p / (E + 1); b0 < a.count_blocks; b0 += 8 * per) {
      int part[8];
#pragma unroll
      for (int b = 0; b < 8; ++b) part[b] = partial[(b0 + b * per < a.count_blocks ? b0 + b * per : b0) * (E + 1) + e];
#pragma unroll
      for (int b = 0; b < 8; ++b) n += b0 + b * per < a.count_blocks ? part[b] : 0;
    }
    if (n != 0) atomicAdd(bins + e, n);
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e < E; e += blockDim.x)
      if (bins[e] != 0) atomicAdd(a.counts + e, bins[e]);  // whole numbers: in any order
  const float sum = take_rows<D, L, NV>(a, bins, first, last, blockDim.x / L, scale, x, valid);
  const double mine = block_sum(bins[E] > 0 ? static_cast<double>(sum) / bins[E] : 0.0, waves);
  const int blocks = a.blocks * a.sequences;
  if (threadIdx.x == 0) {
    __hip_atomic_store(a.sums + static_cast<int64_t>(s) * a.blocks + blockIdx.x, mine, __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the sum is in memory
    last_block = __hip_atomic_fetch_add(a.done, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == blocks - 1;
    asm volatile("" ::: "memory");
  }
  __syncthreads();
  if (!last_block) return;
  double total = 0.0;
  for (int b = threadIdx.x; b < blocks; b += blockDim.x)
    total += __hip_atomic_load(a.sums + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  total = block_sum(total, waves);
  if (threadIdx.x == 0) *a.loss = static_cast<float>(total * alpha);
}

template <int D, int L, int NV>
void launch_rows(const BalanceArgs& a, hipStream_t s) {
  const bool small = a.count_blocks == 0;
  const dim3 grid(a.blocks, small ? 1 : a.sequences), block(small ? kSmallThreads : kThreads / NV);
  hipLaunchKernelGGL((balance_rows_kernel<D, L, NV>), grid, block, 0, s, a);
}

// Lanes of a row: the fewest that hold it, 8 elements each.
int lanes_of(int experts) {
  int lanes = 1;
  while (lanes < 64 && lanes * kElems < experts) lanes *= 2;
  return lanes;
}

template <int D>
hipError_t launch_rows(const BalanceArgs& a, hipStream_t s) {
  switch (lanes_of(a.experts)) {
    case 1: launch_rows<D, 1, 1>(a, s); break;
    case 2: launch_rows<D, 2, 1>(a, s); break;
    case 4: launch_rows<D, 4, 1>(a, s); break;
    case 8: launch_rows<D, 8, 1>(a, s); break;
    case 16: launch_rows<D, 16, 1>(a, s); break;
    case 32: launch_rows<D, 32, 1>(a, s); break;
    default:
      if (a.experts <= 64 * kElems) {
        launch_rows<D, 64, 1>(a, s);
      } else {
        launch_rows<D, 64, 2>(a, s);
      }
      break;
  }
  return hipGetLastError();
}

struct Plan {
  int count_blocks, blocks;  // of a sequence; count_blocks 0: one block in all
};

Plan plan_of(int sequences, int tokens, int experts, int top) {
  const int64_t rows = static_cast<int64_t>(sequences) * tokens;
  const int lanes = lanes_of(experts);
  // one block / two launches, us: 7 x 8, top 2, 5.6 / 8.7; 512 x 8, top 2, 5.7 / 9.4; 128 x 64,
  // top 6, 7.4 / 10.6; 32 x 256, top 8, 8.1 / 11.5; 16 x 1024, top 8, 11.8 / 12.1; past the bounds
  // 2048 x 8, top 1, 9.3 / 10.4; 512 x 64, top 2, 15.8 / 10.9; 32 x 1024, top 8, 17.4 / 12.2.
  // Sequences are taken one after the other: 2 x 64 x 64, top 6, 9.2 / 9.6, but 4 x 8 x 64
  // 12.8 / 9.5; 8 x 8 x 8, top 2, 19.3 / 9.5
  if (rows * top <= 4 * kSmallThreads && rows <= 4 * kSmallThreads / lanes && sequences <= 4) return Plan{0, 1};
  const int per = (experts > 64 * kElems ? kThreads / 2 : kThreads) / lanes;  // rows of a block at a time
  const int64_t entries = static_cast<int64_t>(tokens) * top;
  int64_t count_blocks = (entries + 2047) / 2048;  // two rounds of loads of a thread
  // and few enough that every block can add them up (at most 8 / 16 / 48 a sequence, us, top
  // 6, bf16): 32768 x 64 17.0 / 16.0 / 15.0, 131072 x 64 33 / 26 / 21, 2 x 65536 x 64 26 / 23 / 20, 7 x
  // 32768 x 64 26.6 / 25.6 / 25.3, 8 x 32768 x 64 27.6 / 26.8 / 26.4, 16 x 16384 x 64 26.5 / 26.2 /
  // 27.6; up to 8192 tokens a sequence within 0.5 of each other
  const int64_t limit = sequences < 8 ? 48 : 8;
  count_blocks = count_blocks > limit ? limit : count_blocks;
  int64_t blocks = (tokens + per - 1) / per;
  // one block a compute unit: all of them count themselves as done at one address.
  // 1024 blocks of a quarter of the threads take 25 us for 32768 x 256 bf16 where these
  // take 18, and 19 instead of 11 for 16 x 2049 x 61
  const int64_t most = sequences < 256 ? 256 / sequences : 1;
  blocks = blocks > most ? most : blocks;
  return Plan{static_cast<int>(count_blocks), static_cast<int>(blocks)};
}

int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }
int64_t partial_bytes(const Plan& p, int sequences, int experts) {
  return up256(static_cast<int64_t>(sequences) * p.count_blocks * (experts + 1) * 4);
}
int64_t sums_bytes(const Plan& p, int sequences) { return up256(static_cast<int64_t>(sequences) * p.blocks * 8); }

bool sizes_ok(int sequences, int tokens, int experts, int top) {
  return sequences >= 1 && tokens >= 1 && experts >= 1 && top >= 1 && experts <= kMaxExperts && sequences <= 65535 &&
         static_cast<int64_t>(sequences) * tokens < (static_cast<int64_t>(1) << 31) &&
         static_cast<int64_t>(sequences) * tokens * top < (static_cast<int64_t>(1) << 31);
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

size_t muon_expert_balance_workspace_size(int sequences, int tokens, int experts, int top) {
  if (!sizes_ok(sequences, tokens, experts, top)) return 0;
  const Plan p = plan_of(sequences, tokens, experts, top);
  return static_cast<size_t>(partial_bytes(p, sequences, experts) + sums_bytes(p, sequences) + 256);
}

muon_status muon_expert_balance(int sequences, int tokens, int experts, int top, const void* logits, muon_dtype z_dtype,
                                int64_t row_stride, const void* index, int index_bits, const uint8_t* mask,
                                muon_expert_score score, double coefficient, const float* grad_scale, float* loss,
                                int32_t* counts, void* grad, int accumulate, void* workspace, size_t ws_bytes,
                                void* stream) {
  const size_t need = muon_expert_balance_workspace_size(sequences, tokens, experts, top);
  if (need == 0) return MUON_ERR_INVALID_ARG;
  if (z_dtype != MUON_F32 && z_dtype != MUON_BF16 && z_dtype != MUON_F16) return MUON_ERR_INVALID_ARG;
  if (logits == nullptr || index == nullptr || loss == nullptr || counts == nullptr || row_stride < 0 ||
      (index_bits != 32 && index_bits != 64) || (score != MUON_SOFTMAX && score != MUON_SIGMOID) ||
      (accumulate != 0 && accumulate != 1) || (accumulate == 1 && grad == nullptr) || grad == logits)
    return MUON_ERR_INVALID_ARG;
  const float alpha = static_cast<float>(coefficient / sequences);
  if (!(coefficient - coefficient == 0.0) || !(alpha - alpha == 0.0f)) return MUON_ERR_INVALID_ARG;  // not finite
  if (workspace == nullptr || ws_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return MUON_ERR_WORKSPACE;
  const Plan p = plan_of(sequences, tokens, experts, top);
  char* ws = static_cast<char*>(workspace);
  BalanceArgs a;
  a.sequences = sequences;
  a.tokens = tokens;
  a.experts = experts;
  a.top = top;
  a.logits = logits;
  a.stride = row_stride;
  a.index = index;
  a.wide = index_bits == 64;
  a.mask = mask;
  a.sigmoid = score == MUON_SIGMOID;
  a.coefficient = alpha;
  a.grad_scale = grad_scale;
  a.loss = loss;
  a.counts = counts;
  a.grad = grad;
  a.accumulate = accumulate;
  a.count_blocks = p.count_blocks;
  a.blocks = p.blocks;
  a.partial = reinterpret_cast<int32_t*>(ws);
  a.sums = reinterpret_cast<double*>(ws + partial_bytes(p, sequences, experts));
  a.done = reinterpret_cast<int32_t*>(ws + partial_bytes(p, sequences, experts) + sums_bytes(p, sequences));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const double rows = static_cast<double>(sequences) * tokens, size = z_dtype == MUON_F32 ? 4.0 : 2.0;
  if (p.count_blocks > 0 &&
      traced_launch(s, "balance_count_kernel", "expert_counts", 0.0, rows * top * index_bits / 8, [&] {
        hipLaunchKernelGGL(balance_count_kernel, dim3(a.count_blocks, sequences), dim3(kCountThreads), 0, s, a);
        return hipGetLastError();
      }) != hipSuccess)
    return MUON_ERR_HIP;
  if (traced_launch(s, "balance_rows_kernel", "expert_balance", 8.0 * rows * experts,
                    rows * experts * size * (grad == nullptr ? 1.0 : accumulate ? 3.0 : 2.0), [&] {
                      switch (z_dtype) {
                        case MUON_F32: return launch_rows<kF32>(a, s);
                        case MUON_BF16: return launch_rows<kBF16>(a, s);
                        default: return launch_rows<kF16>(a, s);
                      }
                    }) != hipSuccess)
    return MUON_ERR_HIP;
  return MUON_OK;
}

}  // extern "C"

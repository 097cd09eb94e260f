// C = A B^T (+ C) of two matrices in the 8-bit code (see muon_fp8_gemm.h for the
// tiles), with a kernel of its own for at most 16 rows of A.
#include "muon_fp8_gemm.h"

namespace muon {
namespace fp8 {
namespace {

template <class T, int FA, bool EXACT>
__global__ __launch_bounds__(256, kBlocksPerCU<T>) void fp8_tile_gemm_kernel(Fp8GemmArgs a, int tm, int tn, int tiles) {
  FP8_LDS(T);
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)), lane = threadIdx.x & 63;
  take_tiles<T, FA, EXACT>(
      lds,
      [&](int* id, Work* t) {
        if (*id >= tiles) return false;
        int outer, ti, tj;
        tile_of(*id, tiles, tm, tn, &outer, &ti, &tj);
        const int b = outer / a.pieces, piece = outer - b * a.pieces;
        t->A = Operand{a.A[b], a.As[b], ti * T::TM, static_cast<uint32_t>(a.m), a.units};
        t->B = Operand{a.B[b], a.Bs[b], tj * T::TN, static_cast<uint32_t>(a.n), a.units};
        t->ub = piece * a.piece_units;
        t->ue = t->ub + a.piece_units < a.units ? t->ub + a.piece_units : a.units;
        t->sums = a.pieces > 1;
        t->C = t->sums ? a.partial + (static_cast<int64_t>(piece) * a.batch + b) * a.m * a.n : a.C[b];
        t->rows = a.m;
        t->cols = a.n;
        t->add = a.accumulate != 0;
        return true;
      },
      wave, lane);
}

// ---------------------------------------------------------------------------
// The pieces of a product that was split along k, added in their order.  Some 4 us
// behind the product, most of it the launch.
// ---------------------------------------------------------------------------
template <int DC>
__global__ __launch_bounds__(256) void fp8_join_kernel(Fp8GemmArgs a) {
  const int b = blockIdx.z;
  const int64_t mn = static_cast<int64_t>(a.m) * a.n, step = static_cast<int64_t>(a.batch) * mn;
  const float* part = a.partial + b * mn;
  void* C = a.C[b];
  const bool vec = (mn & 3) == 0 && (reinterpret_cast<uintptr_t>(C) & (DC == kF32 ? 15u : 7u)) == 0;
  for (int64_t at = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4; at < mn;
       at += static_cast<int64_t>(gridDim.x) * 1024) {
    const int left = mn - at < 4 ? static_cast<int>(mn - at) : 4;
    float v[4] = {};
    for (int p = 0; p < a.pieces; ++p) {
      if (vec) {
        const float4 x = *reinterpret_cast<const float4*>(part + p * step + at);
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < left) v[e] += part[p * step + at + e];
      }
    }
    store_quad<DC>(C, at, v, left, vec, a.accumulate);
  }
}

// ---------------------------------------------------------------------------
// At most 16 rows of A (a few tokens against a weight): the codes of B are what
// has to be read.  A wave takes 16 rows of B (a lane 32 bytes of one row; a unit of
// 16 rows is two runs of 1 KB) and every NW-th unit of k, straight from memory into
// registers, and multiplies as kExact does (16x16x32 MFMAs; memory takes longer than
// the conversions).  The block's NW sums are added in LDS, in their order.  Rows of A
// behind the last one repeat it and are not stored.  Bound by memory: 18944 x 3584 codes
// 13.4 us, 5.0 TB/s, 100000 x 4096 78 us, 5.3 (two units ahead of 8 waves; four of 4
// waves 16.7 us, loads past the caches slower).
// ---------------------------------------------------------------------------
constexpr int kFewRows = 16;
constexpr int kUnitsAhead = 2;

template <int FA, int S>
__device__ __forceinline__ f32x4_t few_step(f32x4_t acc, const Frag& a, const Frag& b, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(to_bf16<kE4M3, S>(b, sb), to_bf16<FA, S>(a, sa), acc, 0, 0, 0);
}

template <int NW, int FA>
__global__ __launch_bounds__(64 * NW) void fp8_few_rows_kernel(Fp8GemmArgs a) {
  __shared__ f32x4_t sums[NW][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, b = blockIdx.z;
  const int j0 = blockIdx.x * 16, r = lane & 15, part = lane >> 4;
  const int ra = r < a.m ? r : a.m - 1, rb = j0 + r < a.n ? j0 + r : a.n - 1;
  const int64_t pa = fp8_pitch(a.m), pb = fp8_pitch(a.n);
  const uint4* A = static_cast<const uint4*>(a.A[b]) + (static_cast<int64_t>(part >> 1) * a.m + ra) * 4 + (part & 1) * 2;
  const uint4* B = static_cast<const uint4*>(a.B[b]) + (static_cast<int64_t>(part >> 1) * a.n + rb) * 4 + (part & 1) * 2;
  const uint8_t* As = static_cast<const uint8_t*>(a.As[b]) + ra;
  const uint8_t* Bs = static_cast<const uint8_t*>(a.Bs[b]) + rb;
  f32x4_t acc = {};
  for (int u0 = wave; u0 < a.units; u0 += NW * kUnitsAhead) {
    Frag av[kUnitsAhead], bv[kUnitsAhead];
    uint32_t sa[kUnitsAhead], sb[kUnitsAhead];
#pragma unroll
    for (int k = 0; k < kUnitsAhead; ++k) {
      const int64_t u = u0 + k * NW < a.units ? u0 + k * NW : u0;  // one behind the last unit is not used
      av[k].lo = A[u * 8 * a.m];
      av[k].hi = A[u * 8 * a.m + 1];
      bv[k].lo = B[u * 8 * a.n];
      bv[k].hi = B[u * 8 * a.n + 1];
      sa[k] = As[u * pa];
      sb[k] = Bs[u * pb];
    }
#pragma unroll
    for (int k = 0; k < kUnitsAhead; ++k)
      if (u0 + k * NW < a.units) {
        acc = few_step<FA, 0>(acc, av[k], bv[k], sa[k], sb[k]);
        acc = few_step<FA, 1>(acc, av[k], bv[k], sa[k], sb[k]);
        acc = few_step<FA, 2>(acc, av[k], bv[k], sa[k], sb[k]);
        acc = few_step<FA, 3>(acc, av[k], bv[k], sa[k], sb[k]);
      }
  }
  sums[wave][lane] = acc;
  __syncthreads();
  if (threadIdx.x >= 64) return;
  // lane l: row l % 16 of C, columns 4 (l / 16) .. + 3
  const int j = j0 + 4 * part;
  if (r >= a.m || j >= a.n) return;
  f32x4_t s = sums[0][lane];
#pragma unroll
  for (int q = 1; q < NW; ++q) s += sums[q][lane];
  const float v[4] = {s[0], s[1], s[2], s[3]};
  void* C = a.C[b];
  const bool vec = (a.n & 3) == 0 && (reinterpret_cast<uintptr_t>(C) & (a.c_dtype == kF32 ? 15u : 7u)) == 0;
  const int64_t at = static_cast<int64_t>(r) * a.n + j;
  if (a.c_dtype == kF32) {
    store_quad<kF32>(C, at, v, a.n - j, vec, a.accumulate);
  } else {
    store_quad<kBF16>(C, at, v, a.n - j, vec, a.accumulate);
  }
}

template <class T>
int64_t tiles_of(int batch, int m, int n) {
  return static_cast<int64_t>(ceil_div(m, T::TM)) * ceil_div(n, T::TN) * batch;
}

// Pieces along k of a product in 64 x 128 tiles that leave compute units idle:
// the fewest microseconds of units (two slabs, one block on a compute unit) plus, for
// more than one piece, the joining launch and the partial sums' way through memory (8
// bytes an element and piece at 6 TB/s).  One time of a unit stands for both types (0.55
// for fp32 results, 0.33 for bf16): the plan, like the workspace query, does not know C's
// type.  So fp32 results always gain, and bf16 ones lose where a split saves little.
// Split / whole, bf16 and fp32 results (us): 64 x 3584 x 18944 19 / 51, 21 / 86; 64 x 2048 x
// 7168 14.5 / 19.2, 15.8 / 35; 64 x 4096 x 4096 13.6 / 12.8, 14.8 / 22; 200 x 3584 x 3584 14.3 /
// 11.9, 18.4 / 20.4; 93 x 1875 x 2233 bf16 12.0 / 9.0.
void split_k(int64_t tiles, int units, double elements, Fp8Plan* p) {
  constexpr int kMinUnits = 4;  // of a piece
  double best = 0.0;
  for (int q = 1; q * tiles <= kCUs && (q == 1 || units / q >= kMinUnits); ++q) {
    const double us = ceil_div(units, q) * 0.52 + (q > 1 ? 4.5 + q * elements * 8.0 / 6e6 : 0.0);
    if (q == 1 || us < best) {
      best = us;
      p->piece_units = ceil_div(units, q);
      p->pieces = ceil_div(units, p->piece_units);
    }
  }
}

template <class T>
void launch_tiles(const Fp8GemmArgs& a, hipStream_t s) {
  const int tm = ceil_div(a.m, T::TM), tn = ceil_div(a.n, T::TN);
  const int tiles = tm * tn * a.batch * a.pieces;
  const dim3 grid(blocks_of<T>(tiles)), block(256);
  const bool e4m3 = a.a_format == kE4M3;
  if (a.c_dtype == kF32) {
    auto* kernel = e4m3 ? fp8_tile_gemm_kernel<T, kE4M3, kExact> : fp8_tile_gemm_kernel<T, kE5M2, kExact>;
    hipLaunchKernelGGL(kernel, grid, block, 0, s, a, tm, tn, tiles);
  } else {
    auto* kernel = e4m3 ? fp8_tile_gemm_kernel<T, kE4M3, kFast> : fp8_tile_gemm_kernel<T, kE5M2, kFast>;
    hipLaunchKernelGGL(kernel, grid, block, 0, s, a, tm, tn, tiles);
  }
}

template <int NW>
void launch_few(const Fp8GemmArgs& a, hipStream_t s) {
  const dim3 grid(ceil_div(a.n, 16), 1, a.batch), block(64 * NW);
  if (a.a_format == kE4M3) {
    hipLaunchKernelGGL((fp8_few_rows_kernel<NW, kE4M3>), grid, block, 0, s, a);
  } else {
    hipLaunchKernelGGL((fp8_few_rows_kernel<NW, kE5M2>), grid, block, 0, s, a);
  }
}

}  // namespace
}  // namespace fp8

using namespace fp8;

// Which kernel, by the times measured (us, bf16 results; m x n x k):
//   few rows   up to the 16 of its MFMA: 1 x 18944 x 3584 13.6, in 64 x 128 tiles 13.9; 1 x
//              3584 x 18944 12.8 and 17.4; 16 x 18944 x 3584 12.8 and 13.4
//   64 x 128   where one round of them leaves nothing for larger ones: 512 x 4096 x 4096
//              14.9, in 128 x 128 tiles 15.8, fp32 23.5 and 29.6; not 576 rows 24.0 and 16.3,
//              fp32 32 and 30
//   128 x 128 or 256 x 256, whichever takes less (big_tiles_pay).  Measured: 8192 x 8192 x
//              8192 451 / 394, 3584 x 7168 x 8192 189 / 182, 4096 x 3584 x 18944 240 / 204; 4864 x
//              4608 x 8192 163 / 180, 5000 x 6656 x 2048 71 / 92, 3584 x 7168 x 2048 55 / 63,
//              8192 x 7168 x 1024 66 / 87, 2048 x 4096 x 8192 59 / 82.  Near the border either may
//              lead by some percent, by card (8192 x 7168 x 3584, in 256 x 256: 186 / 195, on
//              another 199 / 193).  Of 46 products of random sizes, in either type, what is
//              chosen takes 2 % over the best at most in nine of ten, 6 % at the worst; of 24
//              of up to 1500 rows 7 and 33 % (bf16 ones that are split, above).
// None of the rules knows whether C is added to.  bf16 C in 256 x 256 tiles is read in
// place then: += 8192 x 8192 x 2048 141 / 178 (fp32 268 / 285), 8192 x 8192 x 8192 461 / 452.
Fp8Plan fp8_plan(int batch, int m, int n, int k) {
  const int units = static_cast<int>(fp8_units(k));
  Fp8Plan p{kF8FewRows, 1, units, 0};
  if (m <= kFewRows) return p;
  const int64_t low = tiles_of<Low>(batch, m, n);
  if (low <= kCUs) {
    p.kind = kF8Low;
    const double elements = static_cast<double>(batch) * m * n;
    split_k(low, units, elements, &p);
    if (p.pieces > 1) p.bytes = static_cast<size_t>(p.pieces) * batch * m * n * sizeof(float);
    return p;
  }
  const double big = static_cast<double>(tiles_of<Big>(batch, m, n)), mid = static_cast<double>(tiles_of<Mid>(batch, m, n));
  p.kind = big_tiles_pay(big, big, mid, units, 1.0) ? kF8Big : kF8Mid;
  return p;
}

hipError_t launch_fp8_gemm(const Fp8GemmArgs& a, Fp8Kind kind, hipStream_t s) {
  switch (kind) {
    case kF8Big: launch_tiles<Big>(a, s); break;
    case kF8Mid: launch_tiles<Mid>(a, s); break;
    case kF8Low: launch_tiles<Low>(a, s); break;
    default:
      // 8 waves of a block and several blocks on a compute unit, or 16 where there is one
      // and k is long (8 / 16 waves, us): 1 x 18944 x 3584 13.1 / 15.1, 16 x 18944 x 3584 12.7 /
      // 15.4; 1 x 2048 x 16384 9.7 / 8.5, 1 x 3584 x 18944 12.5 / 12.4, 1 x 4096 x 8192 6.9 both
      if (a.units >= 64 && ceil_div(a.n, 16) * a.batch <= kCUs) {
        launch_few<16>(a, s);
      } else {
        launch_few<8>(a, s);
      }
      break;
  }
  return hipGetLastError();
}

hipError_t launch_fp8_join(const Fp8GemmArgs& a, hipStream_t s) {
  const int64_t blocks = (static_cast<int64_t>(a.m) * a.n + 1023) / 1024;
  const dim3 grid(static_cast<uint32_t>(blocks < 4096 ? blocks : 4096), 1, a.batch), block(256);
  if (a.c_dtype == kF32) {
    hipLaunchKernelGGL(fp8_join_kernel<kF32>, grid, block, 0, s, a);
  } else {
    hipLaunchKernelGGL(fp8_join_kernel<kBF16>, grid, block, 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace muon

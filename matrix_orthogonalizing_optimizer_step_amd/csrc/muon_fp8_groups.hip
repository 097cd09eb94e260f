// The products of 8-bit codes over groups with row counts on the device (the
// experts of a mixture): rows of A and C in groups, each with its own B; and k in
// groups, each with its own C.
#include "muon_fp8_gemm.h"

namespace muon {
namespace fp8 {
namespace {

// The grid holds as many row tiles as any counts can need; a block finds its group
// by a scan of the counts, and those behind the last tile end at once.
template <class T, int FA, bool EXACT>
__global__ __launch_bounds__(256, kBlocksPerCU<T>) void fp8_row_groups_kernel(Fp8RowGroupArgs a, int tn) {
  FP8_LDS(T);
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)), lane = threadIdx.x & 63;
  const RowTiles<T::TM> tiles{a.counts, a.groups, a.m, a.first, a.first + a.count + a.clear};
  // consecutive ids go to the 8 XCDs in turn: each gets a contiguous range of tiles
  const int total = tiles.all(lane) * tn, q = total >> 3, rest = total & 7, x = blockIdx.x & 7, at = blockIdx.x >> 3;
  if (at >= q + (x < rest ? 1 : 0)) return;
  const RowTile g = tiles.of(x * q + (x < rest ? x : rest) + at, tn, lane);
  if (g.group < 0) return;
  // down columns of 4 tile rows of the group, as in tile_of
  constexpr int kGroup = 4;
  const int band = g.tile / (kGroup * tn), top = band * kGroup, h = g.tiles - top < kGroup ? g.tiles - top : kGroup;
  const int t = g.tile - band * kGroup * tn;
  const int i0 = g.begin + (top + t % h) * T::TM, j0 = t / h * T::TN;
  if (g.group == a.groups) {  // rows behind the last group
    const int rows = g.end - i0 < T::TM ? g.end - i0 : T::TM, cols = a.n - j0 < T::TN ? a.n - j0 : T::TN;
    for (int p = threadIdx.x; p < rows * cols; p += 256)
      store_from_f32(a.C, static_cast<int64_t>(i0 + p / cols) * a.n + j0 + p % cols, a.c_dtype, 0.0f);
    return;
  }
  const int e = g.group - a.first;
  const Source A{a.A, 0, static_cast<uint32_t>(a.m)};
  const Source B{a.B[e], 0, static_cast<uint32_t>(a.n)};
  f32x16_t acc[T::FN][T::FM] = {};
  tile_product<T, FA, EXACT>(acc, lds, A, B, a.As, a.Bs[e], i0, j0, 0, a.units, a.units, wave, lane);
  const int i = i0 + T::FM * 32 * (wave / T::WN), j = j0 + T::FN * 32 * (wave % T::WN);
  typename T::Stage& stage = wave == 0 ? s0 : wave == 1 ? s1 : wave == 2 ? s2 : s3;
  store_product<T, EXACT>(a.C, acc, stage, i, j, g.end, a.n, lane, a.accumulate);
}

template <class T, int FA, bool EXACT>
__global__ __launch_bounds__(256, kBlocksPerCU<T>) void fp8_k_groups_kernel(Fp8KGroupArgs a, int tm, int tn) {
  FP8_LDS(T);
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)), lane = threadIdx.x & 63;
  int e, ti, tj, ub, ue;
  tile_of(blockIdx.x, gridDim.x, tm, tn, &e, &ti, &tj);
  group_units(a.counts, a.groups, a.rows, a.first + e, a.units, lane, &ub, &ue);
  const int i0 = ti * T::TM, j0 = tj * T::TN;
  const Source A{a.A, 0, static_cast<uint32_t>(a.m)};
  const Source B{a.B, 0, static_cast<uint32_t>(a.n)};
  f32x16_t acc[T::FN][T::FM] = {};
  tile_product<T, FA, EXACT>(acc, lds, A, B, a.As, a.Bs, i0, j0, ub, ue, a.units, wave, lane);
  const int i = i0 + T::FM * 32 * (wave / T::WN), j = j0 + T::FN * 32 * (wave % T::WN);
  typename T::Stage& stage = wave == 0 ? s0 : wave == 1 ? s1 : wave == 2 ? s2 : s3;
  store_product<T, EXACT>(a.C[e], acc, stage, i, j, a.m, a.n, lane, a.accumulate);
}

template <class T>
void launch_rows(const Fp8RowGroupArgs& a, hipStream_t s) {
  const int tn = ceil_div(a.n, T::TN);
  // whole tiles of all rows, and one that is not full for each group and for the rest
  const int64_t tm = a.m / T::TM + a.count + a.clear;
  const dim3 grid(static_cast<uint32_t>(tm * tn)), block(256);
  const bool e4m3 = a.a_format == kE4M3;
  if (a.c_dtype == kF32) {
    auto* kernel = e4m3 ? fp8_row_groups_kernel<T, kE4M3, kExact> : fp8_row_groups_kernel<T, kE5M2, kExact>;
    hipLaunchKernelGGL(kernel, grid, block, 0, s, a, tn);
  } else {
    auto* kernel = e4m3 ? fp8_row_groups_kernel<T, kE4M3, kFast> : fp8_row_groups_kernel<T, kE5M2, kFast>;
    hipLaunchKernelGGL(kernel, grid, block, 0, s, a, tn);
  }
}

template <class T>
void launch_k(const Fp8KGroupArgs& a, hipStream_t s) {
  const int tm = ceil_div(a.m, T::TM), tn = ceil_div(a.n, T::TN);
  const dim3 grid(static_cast<uint32_t>(tm) * tn * a.count), block(256);
  const bool e4m3 = a.a_format == kE4M3;
  if (a.c_dtype == kF32) {
    auto* kernel = e4m3 ? fp8_k_groups_kernel<T, kE4M3, kExact> : fp8_k_groups_kernel<T, kE5M2, kExact>;
    hipLaunchKernelGGL(kernel, grid, block, 0, s, a, tm, tn);
  } else {
    auto* kernel = e4m3 ? fp8_k_groups_kernel<T, kE4M3, kFast> : fp8_k_groups_kernel<T, kE5M2, kFast>;
    hipLaunchKernelGGL(kernel, grid, block, 0, s, a, tm, tn);
  }
}

}  // namespace
}  // namespace fp8

using namespace fp8;

Fp8Kind fp8_row_group_kind(int groups, int m, int n) {
  const int64_t mean = m / groups;
  return mean >= 192 && n >= 192 ? kF8Big : mean >= 48 ? kF8Mid : kF8Low;
}

hipError_t launch_fp8_row_groups(const Fp8RowGroupArgs& a, Fp8Kind kind, hipStream_t s) {
  switch (kind) {
    case kF8Big: launch_rows<Big>(a, s); break;
    case kF8Mid: launch_rows<Mid>(a, s); break;
    default: launch_rows<Low>(a, s); break;
  }
  return hipGetLastError();
}

Fp8Kind fp8_k_group_kind(int groups, int m, int n) {
  const int64_t big = static_cast<int64_t>(ceil_div(m, Big::TM)) * ceil_div(n, Big::TN) * groups;
  return big >= kCUs ? kF8Big : kF8Mid;
}

hipError_t launch_fp8_k_groups(const Fp8KGroupArgs& a, Fp8Kind kind, hipStream_t s) {
  switch (kind) {
    case kF8Big: launch_k<Big>(a, s); break;
    default: launch_k<Mid>(a, s); break;
  }
  return hipGetLastError();
}

}  // namespace muon

// The products of 8-bit codes over groups with row counts on the device (the
// experts of a mixture): rows of A and C in groups, each with its own B; and k in
// groups, each with its own C.
#include "muon_fp8_gemm.h"

namespace muon {
namespace fp8 {
namespace {

// Counts of a launch's groups (at most `rows` each, the rest as one more group) and
// the rows before them, in LDS: a block that stays looks for its next tile while its
// loads are under way, and must not wait for other ones.
struct Counts {
  int32_t rows[kF8Groups + 1];
  int before;
};

__device__ __forceinline__ void read_counts(Counts& c, const int32_t* counts, int groups, int rows, int first, int count) {
  if (threadIdx.x <= kF8Groups) {
    const int g = static_cast<int>(threadIdx.x);
    c.rows[g] = g <= count ? group_count(counts, first + g, groups, rows) : 0;
  }
  if (threadIdx.x < 64) {
    int n = 0;
    for (int g = threadIdx.x; g < first; g += 64) n += group_count(counts, g, groups, rows);
    n = wave_scan(n);
    if (threadIdx.x == 63) c.before = n;
  }
  __syncthreads();
}

// As many row tiles as there are at most are launched; a block finds its group by a
// scan of the counts, and those behind the last tile end at once.
template <class T, int FA, bool EXACT>
__global__ __launch_bounds__(256, kBlocksPerCU<T>) void fp8_row_groups_kernel(Fp8RowGroupArgs a, int tn) {
  FP8_LDS(T);
  __shared__ Counts counts;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)), lane = threadIdx.x & 63;
  read_counts(counts, a.counts, a.groups, a.m, a.first, a.count);
  const auto count = [&](int g) { return counts.rows[g]; };
  const RowTiles<T::TM, decltype(count)> row_tiles{count, a.m, a.count, __builtin_amdgcn_readfirstlane(counts.before)};
  if (a.clear) {  // rows behind the last group
    int used = counts.before;
    for (int g = 0; g < a.count; ++g) used += counts.rows[g];
    const int64_t row = static_cast<int64_t>(a.n) * (EXACT ? 4 : 2);
    if (used < a.m) clear_bytes(static_cast<char*>(a.C) + used * row, (a.m - used) * row);
  }
  // consecutive ids go to the 8 XCDs in turn: each gets a contiguous range of tiles
  const int total = row_tiles.all(lane) * tn, q = total >> 3, rest = total & 7;
  take_tiles<T, FA, EXACT>(
      lds,
      [&](int* id, Work* t) {
        const int x = *id & 7, at = *id >> 3;
        if (at >= q + (x < rest ? 1 : 0)) return false;
        const RowTile g = row_tiles.of(x * q + (x < rest ? x : rest) + at, tn, lane);
        int ti, tj;
        tile_in_bands(g.tile, g.tiles, tn, &ti, &tj);
        const int e = g.group;
        t->A = Operand{a.A, a.As, g.begin + ti * T::TM, static_cast<uint32_t>(a.m), a.units};
        t->B = Operand{a.B[e], a.Bs[e], tj * T::TN, static_cast<uint32_t>(a.n), a.units};
        t->ub = 0;
        t->ue = a.units;
        t->sums = false;
        t->C = a.C;
        t->rows = g.end;
        t->cols = a.n;
        t->add = a.accumulate != 0;
        return true;
      },
      wave, lane);
}

template <class T, int FA, bool EXACT>
__global__ __launch_bounds__(256, kBlocksPerCU<T>) void fp8_k_groups_kernel(Fp8KGroupArgs a, int tm, int tn, int ids) {
  FP8_LDS(T);
  __shared__ Counts counts;
  __shared__ int units[kF8Groups + 1];  // before each group
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)), lane = threadIdx.x & 63;
  read_counts(counts, a.counts, a.groups, a.rows, a.first, a.count);
  if (threadIdx.x < 64) {
    int row = 0, n = 0;  // up to the group
    for (int g0 = -a.first; g0 <= a.count; g0 += 64) {
      const int g = g0 + lane;
      const int c = g >= a.count ? 0 : g >= 0 ? counts.rows[g] : group_count(a.counts, a.first + g, a.groups, a.rows);
      const int upto = row + wave_scan(c);
      const int begin = upto - c < a.rows ? upto - c : a.rows, end = upto < a.rows ? upto : a.rows;
      const int mine = (end - begin + kF8Unit - 1) / kF8Unit, sum = n + wave_scan(mine);
      if (g >= 0 && g <= a.count) units[g] = sum - mine < a.units ? sum - mine : a.units;
      row = __builtin_amdgcn_readlane(upto, 63);
      n = __builtin_amdgcn_readlane(sum, 63);
    }
  }
  __syncthreads();
  // consecutive ids go to the 8 XCDs in turn: each gets a contiguous eighth of every
  // group's tiles, since groups take very different times (with whole groups to an
  // XCD, 16 of 2048 x 7168 with 8190 rows in all took 524 us, so 387)
  const int per = tm * tn, share = (per + 7) >> 3;
  if (!a.accumulate)
    for (int e = 0; e < a.count; ++e)
      if (units[e] == units[e + 1]) clear_bytes(a.C[e], static_cast<int64_t>(a.m) * a.n * (EXACT ? 4 : 2));
  take_tiles<T, FA, EXACT>(
      lds,
      [&](int* id, Work* t) {
        for (; *id < ids; *id += gridDim.x) {
          const int at = *id >> 3, e = at / share, tile = (*id & 7) * share + at - e * share;
          t->ub = __builtin_amdgcn_readfirstlane(units[e]);
          t->ue = __builtin_amdgcn_readfirstlane(units[e + 1]);
          if (tile >= per || t->ub == t->ue) continue;  // behind the last eighth's end, or without rows
          int ti, tj;
          tile_in_bands(tile, tm, tn, &ti, &tj);
          t->A = Operand{a.A, a.As, ti * T::TM, static_cast<uint32_t>(a.m), a.units};
          t->B = Operand{a.B, a.Bs, tj * T::TN, static_cast<uint32_t>(a.n), a.units};
          t->sums = false;
          t->C = a.C[e];
          t->rows = a.m;
          t->cols = a.n;
          t->add = a.accumulate != 0;
          return true;
        }
        return false;
      },
      wave, lane);
}

template <class T>
void launch_rows(const Fp8RowGroupArgs& a, hipStream_t s) {
  const int tn = ceil_div(a.n, T::TN);
  // whole tiles of all rows, and one that is not full for each group and for the rest
  const int64_t tm = a.m / T::TM + a.count + a.clear;
  const dim3 grid(blocks_of<T>(tm * tn)), block(256);
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
  const int ids = 8 * ((tm * tn + 7) / 8) * a.count;
  const dim3 grid(blocks_of<T>(ids)), block(256);
  const bool e4m3 = a.a_format == kE4M3;
  if (a.c_dtype == kF32) {
    auto* kernel = e4m3 ? fp8_k_groups_kernel<T, kE4M3, kExact> : fp8_k_groups_kernel<T, kE5M2, kExact>;
    hipLaunchKernelGGL(kernel, grid, block, 0, s, a, tm, tn, ids);
  } else {
    auto* kernel = e4m3 ? fp8_k_groups_kernel<T, kE4M3, kFast> : fp8_k_groups_kernel<T, kE5M2, kFast>;
    hipLaunchKernelGGL(kernel, grid, block, 0, s, a, tm, tn, ids);
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
    case kF8Big: launch_k<Staying>(a, s); break;
    default: launch_k<Mid>(a, s); break;
  }
  return hipGetLastError();
}

}  // namespace muon

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
// scan of the counts, and those behind the last tile end at once.  Few rows are bound by
// the weights: 24 rows, 64 groups of 2048 x 7168 62 to 65 us, 5.0 TB/s.  Many are bound by
// power and by tiles that are not full: 16380 rows 282 us, 1.71 PFLOP/s; with as many rows in
// every group, so that all tiles are full, 226.
template <class T, int FA, bool EXACT>
__global__ __launch_bounds__(256, kBlocksPerCU<T>) void fp8_row_groups_kernel(Fp8RowGroupArgs a, int tn) {
  FP8_LDS(T);
  __shared__ Counts counts;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)), lane = threadIdx.x & 63;
  read_counts(counts, a.counts, a.groups, a.m, a.first, a.count);
  const auto count = [&](int g) { return counts.rows[g]; };
  const RowTiles<T::TM, decltype(count)> row_tiles{count, a.m, a.count, __builtin_amdgcn_readfirstlane(counts.before)};
  if (a.clear) {  // rows behind the last group
    const int mine = (lane < a.count ? counts.rows[lane] : 0) + (lane + 64 < a.count ? counts.rows[lane + 64] : 0);
    const int used = counts.before + __builtin_amdgcn_readlane(wave_scan(mine), 63);
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

// k of a group is its rows, in whole units; the last one is filled up with zero codes.
// Bound by the products (fp32 results: converted codes at half the rate) and, k being
// short, by the results' way to memory: 16 groups of 2048 x 7168, 8190 rows, fp32 334 us
// for 940 MB of results.
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
  // XCD, 16 of 2048 x 7168 with 8190 rows in all took 524 us, so 387 then)
  const int per = tm * tn, share = (per + 7) >> 3;
  if (!a.accumulate)
    for (int e0 = 0; e0 < a.count; e0 += 64)
      for (uint64_t none = __ballot(e0 + lane < a.count && units[e0 + lane] == units[e0 + lane + 1]); none != 0;
           none &= none - 1)
        clear_bytes(a.C[e0 + __builtin_ctzll(none)], static_cast<int64_t>(a.m) * a.n * (EXACT ? 4 : 2));
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
  if (T::kStays || a.c_dtype == kF32) {
    auto* kernel = e4m3 ? fp8_k_groups_kernel<T, kE4M3, kExact> : fp8_k_groups_kernel<T, kE5M2, kExact>;
    hipLaunchKernelGGL(kernel, grid, block, 0, s, a, tm, tn, ids);
  } else if constexpr (!T::kStays) {
    auto* kernel = e4m3 ? fp8_k_groups_kernel<T, kE4M3, kFast> : fp8_k_groups_kernel<T, kE5M2, kFast>;
    hipLaunchKernelGGL(kernel, grid, block, 0, s, a, tm, tn, ids);
  }
}

}  // namespace
}  // namespace fp8

using namespace fp8;

// Which tiles, for rows that are not known here but as a sum: a group's last tile row
// is taken to be half full.  Times in us, 64 x 128 / 128 x 128 / 256 x 256 tiles, rows
// spread unevenly:
//   256 x 256  where they take less than 128 x 128 (big_tiles_pay; these are some 7 %
//              slower here than without groups): 64 groups, n 2048, k 7168, 16380 rows 419 /
//              342 / 282, 32768 rows 769 / 587 / 518; 8 groups, 4096, 2048, 32768 rows 412 /
//              309 / 277; not 16 groups with 8190 rows 170 / 138 / 154, with n 7168 and k 2048
//              195 / 152 / 159, k 1024 111 / 83 / 103; 4 groups, 8192, 4096, 4000 rows 180 /
//              133 / 148
//   128 x 128  from a mean of 96 rows on: those, and 8 groups, 1024 x 1024, 4096 rows 14 /
//              12 / 19
//   64 x 128   for fewer: 64 groups, 24 rows 62 / 70 / 77; 8 groups, 1024 x 1024, 600 rows
//              6.9 / 7.9 / 17; 64 groups, 4000 rows 186 / 193 / 181, fp32 219 / 230 / 307, spread
//              otherwise 183 / 170 / 178, fp32 215 / 208 / 299, with as many in every group
//              173 / 180 / 192, fp32 189 / 205 / 293
// How the rows are spread decides as much as their sum (16 groups of 7168 x 2048 with as
// many in each 155 / 131 in 128 x 128 / 256 x 256).  Of 30 random sizes and spreads what is
// chosen takes the best time at the median, 15 % over it in one of ten, 28 % at the worst
// (few tiles of 128 x 128: 2 groups, 670 rows, 1704 x 5751 fp32 31 / 40 / 109).
Fp8Kind fp8_row_group_kind(int groups, int m, int n, int k) {
  if (m / groups < 96) return kF8Low;
  const int units = static_cast<int>(fp8_units(k));
  const double big = (m / Big::TM + (groups + 1) / 2) * static_cast<double>(ceil_div(n, Big::TN));
  const double mid = (m / Mid::TM + (groups + 1) / 2) * static_cast<double>(ceil_div(n, Mid::TN));
  const double work = static_cast<double>(m) * n / (Big::TM * Big::TN);
  return big_tiles_pay(work, big, mid, units, 1.07) ? kF8Big : kF8Mid;
}

hipError_t launch_fp8_row_groups(const Fp8RowGroupArgs& a, Fp8Kind kind, hipStream_t s) {
  switch (kind) {
    case kF8Big: launch_rows<Big>(a, s); break;
    case kF8Mid: launch_rows<Mid>(a, s); break;
    default: launch_rows<Low>(a, s); break;
  }
  return hipGetLastError();
}

// Which tiles (us, 128 x 128 / 256 x 256 / 256 x 256 by blocks that stay, rows spread
// unevenly):
//   that stay  fp32 results from three rounds of tiles on, where the results' way to
//              memory counts most: 16 groups of 2048 x 7168, 8190 rows 385 / 350 / 334, 64
//              groups, 16380 rows 1220 / 1099 / 1000, 4 groups, 8190 rows 229 / 228 / 212.  A
//              fixed share of the tiles is no good for fewer: 8 groups of 2048 x 2048, 32768
//              rows (two rounds) 233 / 232 / 284, spread otherwise 261 / 246 / 232
//   256 x 256  otherwise from two rounds on, if groups have 192 rows on average: bf16
//              266 / 237, 913 / 802, 125 / 127, 124 / 122
//   128 x 128  for fewer tiles or rows: 16 groups of 1024 x 1024, 2000 rows bf16 15 / 17; 64
//              of 512 x 2048, 1000 rows 50 / 55
// Of 30 random sizes what is chosen takes the best time at the median, 11 % over it in one
// of ten, 35 % at the worst (11 groups of 1383 x 2665, 3084 rows bf16 35 / 47).  The rule does
// not know whether C is added to: bf16 C in 256 x 256 tiles is read in place then (16 groups
// 279 / 436; fp32 424 / 425 / 412).
Fp8Kind fp8_k_group_kind(int groups, int rows, int m, int n, bool fp32) {
  const int64_t big = static_cast<int64_t>(ceil_div(m, Big::TM)) * ceil_div(n, Big::TN) * groups;
  if (fp32 && big >= 3 * kCUs) return kF8Staying;
  return big >= 2 * kCUs && rows / groups >= 192 ? kF8Big : kF8Mid;
}

hipError_t launch_fp8_k_groups(const Fp8KGroupArgs& a, Fp8Kind kind, hipStream_t s) {
  switch (kind) {
    case kF8Staying: launch_k<Staying>(a, s); break;
    case kF8Big: launch_k<Big>(a, s); break;
    default: launch_k<Mid>(a, s); break;
  }
  return hipGetLastError();
}

}  // namespace muon

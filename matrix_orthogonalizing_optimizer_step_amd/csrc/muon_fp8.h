// Layout and element arithmetic of the 8-bit code with a scale for each block of
// 128, shared by its codec and its products, and the device side of row counts.
//
// A row of k elements is cut into units of 128, filled up with zero codes.  A unit
// shares one E8M0 scale byte, which the MFMA takes as an operand, and is stored as
// two pieces of 64 bytes: codes [2 units][rows][64], scales [units][pitch], pitch =
// rows rounded up to 16.  A tile of consecutive rows is then one contiguous run of
// memory for every step of 64 along k.  In a matrix that was coded in 128 x 128
// tiles a tile's byte is repeated for each of its rows, so that a product need not
// know.  Coded along the columns with row counts, each group's rows fill whole
// units: ceil(count / 128) of them, one group behind the other.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muon {

constexpr int kF8Unit = 128;
constexpr int kF8Piece = 64;
constexpr int kF8Line = 16;

enum Fp8Format : int { kE4M3 = 0, kE5M2 = 1 };  // the operand format fields of the MFMA, values of muon_fp8_format

__host__ __device__ inline int64_t fp8_units(int64_t k) { return (k + kF8Unit - 1) / kF8Unit; }
__host__ __device__ inline int64_t fp8_pitch(int64_t rows) { return (rows + kF8Line - 1) / kF8Line * kF8Line; }
// Units that hold `rows` rows in `groups` groups, whatever their counts.
__host__ __device__ inline int64_t fp8_group_units(int64_t rows, int64_t groups) { return (rows + (kF8Unit - 1) * groups) / kF8Unit; }

// Matrices of one launch; their pointers travel with the kernel arguments.
constexpr int kF8Batch = 16;
// Groups whose own pointers one launch takes.
constexpr int kF8Groups = 128;

struct Fp8QuantArgs {
  int x_dtype, format;
  int tile;                  // one scale for 128 x 128 elements
  int rows, cols;
  const int32_t* counts;     // rows of each group, or null (one group)
  int groups;
  const void* X[kF8Batch];
  void* codes[kF8Batch];     // of X, or null
  void* scales[kF8Batch];
  void* codes_t[kF8Batch];   // of X^T, or null
  void* scales_t[kF8Batch];
};
hipError_t launch_fp8_quantize(const Fp8QuantArgs& a, int batch, hipStream_t s);

struct Fp8DequantArgs {
  int rows, cols, format;
  int y_dtype;
  const void* codes[kF8Batch];
  const void* scales[kF8Batch];
  void* Y[kF8Batch];
};
hipError_t launch_fp8_dequantize(const Fp8DequantArgs& a, int batch, hipStream_t s);

// C = A B^T (+ C), for each matrix of a batch.
struct Fp8GemmArgs {
  int batch, m, n, units;
  int a_format, c_dtype;
  int accumulate;
  int pieces, piece_units;      // split along k: units per piece
  float* partial;               // pieces x batch x m x n sums, if pieces > 1
  const void* A[kF8Batch];      // codes of m x k
  const void* As[kF8Batch];     // scales
  const void* B[kF8Batch];      // codes of n x k
  const void* Bs[kF8Batch];
  void* C[kF8Batch];            // m x n, row-major
};

// Rows of A in groups, each with its own B: C[rows of g] = A[rows of g] B_g^T (+ C).
struct Fp8RowGroupArgs {
  int m, n, units;              // m: rows of A and C
  int a_format, c_dtype;
  int accumulate;
  int clear;                    // rows behind the last group become 0
  int groups, first, count;     // all groups; those of this launch
  const int32_t* counts;        // rows of each group, on the device
  const void* A;
  const void* As;
  void* C;
  const void* B[kF8Groups];
  const void* Bs[kF8Groups];
};

// k in groups, each with its own C: C_g = A[:, k of g] B[:, k of g]^T (+ C_g).
struct Fp8KGroupArgs {
  int m, n, units;              // units: fp8_group_units
  int rows;                     // of all groups: the bound of a count
  int a_format, c_dtype;
  int accumulate;
  int groups, first, count;
  const int32_t* counts;
  const void* A;
  const void* As;
  const void* B;
  const void* Bs;
  void* C[kF8Groups];
};

// How a product of one launch is computed.
enum Fp8Kind : int { kF8FewRows = 0, kF8Low, kF8Mid, kF8Big, kF8Staying };
struct Fp8Plan {
  Fp8Kind kind;
  int pieces, piece_units;
  size_t bytes;                 // of partial sums
};
Fp8Plan fp8_plan(int batch, int m, int n, int k);
hipError_t launch_fp8_gemm(const Fp8GemmArgs& a, Fp8Kind kind, hipStream_t s);
hipError_t launch_fp8_join(const Fp8GemmArgs& a, hipStream_t s);  // the pieces' sums into C
Fp8Kind fp8_row_group_kind(int groups, int m, int n, int k);
hipError_t launch_fp8_row_groups(const Fp8RowGroupArgs& a, Fp8Kind kind, hipStream_t s);
Fp8Kind fp8_k_group_kind(int groups, int rows, int m, int n, bool fp32);
hipError_t launch_fp8_k_groups(const Fp8KGroupArgs& a, Fp8Kind kind, hipStream_t s);

// 2^(byte - 127), NaN for byte 255.
__device__ __forceinline__ float fp8_scale_value(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FC00000u : (byte == 0u ? 0x00400000u : byte << 23));
}

// Scale byte of a block from the bits of its largest magnitude: the smallest power
// of two, from 2^-127 on, that leaves it at most 1.75 2^8 (e4m3's 448) or 1.75 2^15
// (e5m2's 57344); 255 for NaN and infinity.
template <int F>
__device__ __forceinline__ uint32_t fp8_scale_byte(uint32_t top_bits) {
  constexpr uint32_t kHigh = F == kE4M3 ? 8u : 15u;
  const uint32_t field = (top_bits >> 23) + ((top_bits & 0x7FFFFFu) > 0x600000u ? 1u : 0u);
  return top_bits >= 0x7F800000u ? 255u : (field > kHigh ? field - kHigh : 0u);
}

// ---------------------------------------------------------------------------
// Groups of consecutive rows, their counts read on the device.  A wave looks at 64
// groups at a time.  Counts under 0 count as 0, and groups end with the last row:
// whatever the counts are, no place is outside the matrix.
// ---------------------------------------------------------------------------
__device__ __forceinline__ int wave_scan(int x) {  // sums over the lanes up to this one
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, true);   // row_shr 1, 2, 4, 8
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // lane 15 of rows 0 and 2 to rows 1 and 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);  // lane 31 to the upper half
  return x;
}

// The count of group g, at most `rows`; group `groups` stands for the rows behind
// the last one.  (The caller has rows x (groups + 1) fit 31 bits: sums do not wrap.)
__device__ __forceinline__ int group_count(const int32_t* counts, int g, int groups, int rows) {
  if (g >= groups) return g == groups ? rows : 0;
  const int c = counts[g];
  return c < 0 ? 0 : (c < rows ? c : rows);
}

struct RowTile {
  int group;       // -1: there is no such tile
  int begin, end;  // rows of the group
  int tile;        // of the group
  int tiles;       // of the group
  int before;      // tiles of the groups before it
};

// Tiles of TM rows of groups 0 .. groups - 1 in order, count(g) rows each from row
// `row0` on.  all: how many there are; of(t): tile t of width 1, or, with `width`
// tiles side by side, the one that the t-th of them all belongs to.
template <int TM, class Count>
struct RowTiles {
  const Count& count;
  int rows, groups, row0;

  __device__ __forceinline__ int all(int lane) const {
    int row = row0, n = 0;
    for (int g0 = 0; g0 < groups; g0 += 64) {
      int upto, tiles, begin, end;
      chunk(g0, lane, row, &upto, &tiles, &begin, &end);
      n += __builtin_amdgcn_readlane(wave_scan(tiles), 63);
      row = __builtin_amdgcn_readlane(upto, 63);
    }
    return n;
  }

  __device__ __forceinline__ RowTile of(int t, int width, int lane) const {
    int row = row0, n = 0;
    for (int g0 = 0; g0 < groups; g0 += 64) {
      int upto, tiles, begin, end;
      chunk(g0, lane, row, &upto, &tiles, &begin, &end);
      const int sum = n + wave_scan(tiles);  // tiles up to this lane's group
      const uint64_t behind = __ballot(t < sum * width);
      if (behind != 0) {
        const int at = __builtin_ctzll(behind);
        RowTile r;
        r.group = g0 + at;
        r.begin = __builtin_amdgcn_readlane(begin, at);
        r.end = __builtin_amdgcn_readlane(end, at);
        r.tiles = __builtin_amdgcn_readlane(tiles, at);
        r.before = __builtin_amdgcn_readlane(sum, at) - r.tiles;
        r.tile = t - r.before * width;
        return r;
      }
      n = __builtin_amdgcn_readlane(sum, 63);
      row = __builtin_amdgcn_readlane(upto, 63);
    }
    return RowTile{-1, 0, 0, 0, 0, 0};
  }

 private:
  // Of groups g0 .. g0 + 63, one a lane: rows up to the group's end, its tiles and place.
  __device__ __forceinline__ void chunk(int g0, int lane, int row, int* upto, int* tiles, int* begin, int* end) const {
    const int g = g0 + lane, c = g < groups ? count(g) : 0;
    *upto = row + wave_scan(c);
    *begin = *upto - c < rows ? *upto - c : rows;
    *end = *upto < rows ? *upto : rows;
    *tiles = (*end - *begin + TM - 1) / TM;
  }
};

}  // namespace muon

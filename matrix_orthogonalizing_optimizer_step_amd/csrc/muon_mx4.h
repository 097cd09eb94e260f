// Layout and element arithmetic of the microscaled 4-bit code, shared by its
// codec and its product.
//
// A matrix of `rows` rows and k columns is cut along each row into units of
// 128 elements, each four blocks of 32 (the last unit is filled up with zero
// codes and scale bytes 0).  Unit u of row r is 64 code bytes at
// (u rows + r) 64 and 4 scale bytes at (u rows + r) 4: a tile of consecutive
// rows is one contiguous piece of memory for every unit, whatever k is, so a
// tile's loads are whole lines and never meet in the same memory channel as
// rows of a power-of-two pitch would.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muon {

constexpr int kMxBlock = 32;
constexpr int kMxUnit = 128;

inline int64_t mx4_units(int64_t k) { return (k + kMxUnit - 1) / kMxUnit; }

// Matrices of one launch; their pointers travel with the kernel arguments.
constexpr int kMxBatch = 16;

struct Mx4QuantArgs {
  int x_dtype;
  int rows, cols;
  const void* X[kMxBatch];
  void* codes[kMxBatch];    // of X, or null
  void* scales[kMxBatch];
  void* codes_t[kMxBatch];  // of X^T, or null
  void* scales_t[kMxBatch];
};
hipError_t launch_mx4_quantize(const Mx4QuantArgs& a, int batch, hipStream_t s);

struct Mx4DequantArgs {
  int rows, cols;
  int y_dtype;
  const void* codes[kMxBatch];
  const void* scales[kMxBatch];
  void* Y[kMxBatch];
};
hipError_t launch_mx4_dequantize(const Mx4DequantArgs& a, int batch, hipStream_t s);

struct Mx4GemmArgs {
  int batch, m, n, k, units;
  int c_dtype;
  int accumulate;               // C += A B^T
  int pieces, piece_units;      // split along k: units per piece
  float* partial;               // pieces x batch x m x n sums, if pieces > 1
  const void* A[kMxBatch];      // codes of m x k
  const void* As[kMxBatch];     // scales
  const void* B[kMxBatch];      // codes of n x k
  const void* Bs[kMxBatch];
  void* C[kMxBatch];            // m x n, row-major
};

// How a product of one launch (at most kMxBatch matrices) is computed.
enum Mx4Kind : int { kMxFewRows = 0, kMxLow, kMxMid, kMxBig };
struct Mx4Plan {
  Mx4Kind kind;
  int pieces, piece_units;
  size_t bytes;                 // of partial sums
};
Mx4Plan mx4_plan(int batch, int m, int n, int k);
hipError_t launch_mx4_gemm(const Mx4GemmArgs& a, Mx4Kind kind, hipStream_t s);
hipError_t launch_mx4_join(const Mx4GemmArgs& a, hipStream_t s);  // the pieces' sums into C

// 2^(byte - 127), NaN for byte 255.
__device__ __forceinline__ float e8m0_to_f32(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FC00000u : (byte == 0u ? 0x00400000u : byte << 23));
}

// Scale byte of a block from the bits of its largest magnitude: two binades
// below it (e2m1's largest value is 6 = 1.5 2^2), 255 for NaN and infinity.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t top_bits) {
  const uint32_t field = top_bits >> 23;
  return field == 255u ? 255u : (field > 2u ? field - 2u : 0u);
}

}  // namespace muon

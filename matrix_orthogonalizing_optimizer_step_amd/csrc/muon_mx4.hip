// The microscaled 4-bit code: blocks of 32 consecutive elements along a row
// share a power of two (one E8M0 byte), each element is an e2m1 float (1 sign,
// 2 exponent, 1 mantissa bit: 0, 1/2, 1, 3/2, 2, 3, 4, 6).  The scale is two
// binades under the block's largest magnitude, elements are rounded to nearest
// even and saturate at 6, as the OCP Microscaling Formats specification (v1.0)
// converts.  Both steps are exact in fp32, so the code of a matrix does not
// depend on how it is computed.
#include "../../include/muon.h"
#include "muon_convert.h"
#include "muon_internal.h"
#include "muon_mx4.h"

namespace muon {
namespace {

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// Rows of odd length start anywhere: loads and stores of 8 and 16 bytes that
// need the alignment of one element only.
typedef u32x2_t u32x2_a2 __attribute__((aligned(2)));
typedef u32x4_t u32x4_a2 __attribute__((aligned(2)));
typedef u32x4_t u32x4_a4 __attribute__((aligned(4)));

template <int D>
__device__ __forceinline__ float half_of(uint32_t w, int upper) {
  const uint16_t h = static_cast<uint16_t>(upper ? w >> 16 : w);
  return D == kBF16 ? bf16_to_f32(h) : f16_to_f32(h);
}

// Scale as the converters take it: its exponent field is the scale byte.
__device__ __forceinline__ float scale_operand(uint32_t byte) { return __uint_as_float(byte << 23); }

// (Macros: a template parameter would drop the pointer type's alignment.)
#define LOAD_VEC(p) (NT ? __builtin_nontemporal_load(p) : *(p))
#define STORE_VEC(p, x)                   \
  do {                                    \
    if constexpr (NT) {                   \
      __builtin_nontemporal_store(x, p);  \
    } else {                              \
      *(p) = x;                           \
    }                                     \
  } while (0)

// Two e2m1 codes of (lo, hi) / scale into byte S of w (nearest even, saturating).
template <int S>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, float lo, float hi, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, lo, hi, scale, S);
}

__device__ __forceinline__ uint32_t code8(const float (&x)[8], float scale) {
  uint32_t w = code_pair<0>(0, x[0], x[1], scale);
  w = code_pair<1>(w, x[2], x[3], scale);
  w = code_pair<2>(w, x[4], x[5], scale);
  return code_pair<3>(w, x[6], x[7], scale);
}

// Largest magnitude of three, NaN if one is NaN.
__device__ __forceinline__ float top3(float a, float b, float c) {
  return __builtin_elementwise_maximum(__builtin_elementwise_maximum(fabsf(a), fabsf(b)), fabsf(c));
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x) {  // of non-negative floats' bits (NaN is largest)
  const uint32_t y = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), CTRL, 0xf, 0xf, true));
  return x > y ? x : y;
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141;  // quad permutations, reversal within 8 lanes

// ---------------------------------------------------------------------------
// Rows of X to or from rows of units: a thread takes 16 bytes of a row of X (8
// 16-bit elements, 4 fp32), so that a wave's access is 1 KB without gaps, for
// kUnitsPerThread units one after the other with all loads out first.
// ---------------------------------------------------------------------------
constexpr int kThreads = 256;
constexpr int kUnitsPerThread = 4;

template <int D>
struct Span {
  static constexpr int kElems = D == kF32 ? 4 : 8;  // of a thread and unit
  static constexpr int kLanes = kMxUnit / kElems;   // threads of a row
  static constexpr int kRows = kThreads / kLanes;   // rows of a block
};

template <int D, bool NT>
__device__ __forceinline__ u32x4_t load_span(const void* X, int64_t at, int left) {
  constexpr int E = Span<D>::kElems;
  if (left >= E) {
    if constexpr (D == kF32) {
      return LOAD_VEC(reinterpret_cast<const u32x4_a4*>(static_cast<const float*>(X) + at));
    } else {
      return LOAD_VEC(reinterpret_cast<const u32x4_a2*>(static_cast<const uint16_t*>(X) + at));
    }
  }
  u32x4_t r = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (e < left) {
      if constexpr (D == kF32) {
        r[e] = static_cast<const uint32_t*>(X)[at + e];
      } else {
        r[e >> 1] |= static_cast<uint32_t>(static_cast<const uint16_t*>(X)[at + e]) << (16 * (e & 1));
      }
    }
  return r;
}

// Codes along rows.  A block of 32 is that of 4 (fp32: 8) neighbouring threads.
template <int D, bool NT>
__global__ __launch_bounds__(kThreads) void mx4_rows_kernel(Mx4QuantArgs a, int units) {
  typedef Span<D> S;
  constexpr int E = S::kElems;
  const int b = blockIdx.z, o = threadIdx.x % S::kLanes;
  const int r = blockIdx.x * S::kRows + static_cast<int>(threadIdx.x) / S::kLanes;
  if (r >= a.rows) return;  // all threads of a row together
  const int u0 = blockIdx.y * kUnitsPerThread;
  const void* X = a.X[b];
  uint8_t* codes = static_cast<uint8_t*>(a.codes[b]);
  uint8_t* scales = static_cast<uint8_t*>(a.scales[b]);
  u32x4_t raw[kUnitsPerThread];
#pragma unroll
  for (int k = 0; k < kUnitsPerThread; ++k) {
    const int c = (u0 + k) * kMxUnit + E * o;
    raw[k] = load_span<D, NT>(X, static_cast<int64_t>(r) * a.cols + c, a.cols - c);
  }
#pragma unroll
  for (int k = 0; k < kUnitsPerThread; ++k) {
    float x[8] = {};
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = D == kF32 ? __uint_as_float(raw[k][e & 3]) : half_of<D>(raw[k][e >> 1], e & 1);
    float most = top3(top3(x[0], x[1], x[2]), x[3], 0.0f);
    if constexpr (E == 8) most = top3(top3(x[4], x[5], x[6]), x[7], most);
    uint32_t top = __float_as_uint(most);
    top = dpp_max<kXor1>(top);
    top = dpp_max<kXor2>(top);
    if constexpr (E == 4) top = dpp_max<kHalfMirror>(top);
    const uint32_t byte = mx4_scale_byte(top);
    const float scale = scale_operand(byte);
    uint32_t w = code_pair<1>(code_pair<0>(0, x[0], x[1], scale), x[2], x[3], scale);
    if constexpr (E == 8) w = code_pair<3>(code_pair<2>(w, x[4], x[5], scale), x[6], x[7], scale);
    w = byte == 255u ? 0u : w;
    if (u0 + k < units) {
      const int64_t line = static_cast<int64_t>(u0 + k) * a.rows + r;
      uint8_t* const c = codes + line * 64 + o * (E / 2);
      if constexpr (E == 8) {
        *reinterpret_cast<uint32_t*>(c) = w;
      } else {
        *reinterpret_cast<uint16_t*>(c) = static_cast<uint16_t>(w);
      }
      if (o % (kMxBlock / E) == 0) scales[line * 4 + o * E / kMxBlock] = static_cast<uint8_t>(byte);
    }
  }
}

// ---------------------------------------------------------------------------
// Codes along columns, or along both, from one read of X: a block of 128
// threads takes a 128 x 128 tile, a thread 32 rows x 4 columns of it in
// registers.  A column's block is then one thread's, a row's block that of 8
// neighbouring lanes.  Each tile's codes are one contiguous 8 KB piece of either
// output; they are put together in LDS and written in whole lines.
// ---------------------------------------------------------------------------
constexpr int kTileThreads = 128;
constexpr int kColPitch = 80;  // bytes of a column's codes in LDS: 64, and 16 against bank conflicts

// The 32 x 4 elements of a thread; rows_left and cols_left of the matrix are
// there, from row 0 and column 0 of them on (none if 0 or less), the others read
// as zero.  `at` is the first element's place.  Where not all are there, the rows
// behind the end read the last one, and the columns over the end the row's last
// four, shifted into place, so that these tiles too have all their loads out at
// once (element by element: 1000x1001 bf16 15.3 us, now 6.3; 4096x4100 28.5, now
// 14.7).
template <int D, bool FULL, bool NT>
__device__ __forceinline__ void load_tile(const void* X, int64_t at, int64_t pitch, int rows_left, int cols_left,
                                          float (&x)[32][4]) {
  if (FULL || pitch >= 4) {
    const int over = FULL || cols_left >= 4 ? 0 : 4 - cols_left;  // columns of the four that are not there
    const int last = rows_left - 1;
    const int64_t from = at - over;
    if constexpr (D == kF32) {
      u32x4_t v[32];
#pragma unroll
      for (int e = 0; e < 32; ++e)
        v[e] = LOAD_VEC(reinterpret_cast<const u32x4_a4*>(static_cast<const float*>(X) + from +
                                                         (FULL || e < last ? e : last) * pitch));
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        if constexpr (!FULL) {
          const u32x4_t none = {0, 0, 0, 0};
          if (over & 1) v[e] = (u32x4_t){v[e][1], v[e][2], v[e][3], 0};
          if (over & 2) v[e] = (u32x4_t){v[e][2], v[e][3], 0, 0};
          if (over >= 4 || e >= rows_left) v[e] = none;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) x[e][c] = __uint_as_float(v[e][c]);
      }
    } else {
      u32x2_t v[32];
#pragma unroll
      for (int e = 0; e < 32; ++e)
        v[e] = LOAD_VEC(reinterpret_cast<const u32x2_a2*>(static_cast<const uint16_t*>(X) + from +
                                                         (FULL || e < last ? e : last) * pitch));
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        if constexpr (!FULL) {
          const uint64_t four = __builtin_bit_cast(uint64_t, v[e]);
          v[e] = __builtin_bit_cast(u32x2_t, over >= 4 || e >= rows_left ? uint64_t{0} : four >> (16 * over));
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) x[e][c] = half_of<D>(v[e][c >> 1], c & 1);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        x[e][c] = e < rows_left && c < cols_left ? load_as_f32(X, at + e * pitch + c, D) : 0.0f;
  }
}

template <int D, bool ROWS, bool NT>
__global__ __launch_bounds__(kTileThreads) void mx4_tile_kernel(Mx4QuantArgs a) {
  __shared__ __align__(16) uint8_t col_code[128 * kColPitch];
  __shared__ __align__(16) uint8_t row_code[ROWS ? 128 * 64 : 16];
  __shared__ __align__(16) uint8_t col_scale[128 * 4];
  __shared__ __align__(16) uint8_t row_scale[ROWS ? 128 * 4 : 16];
  const int b = blockIdx.z, tid = threadIdx.x, h = tid >> 5, l = tid & 31;
  const int i0 = blockIdx.y * 128, j0 = blockIdx.x * 128;
  const int i = i0 + 32 * h, j = j0 + 4 * l;
  const int64_t at = static_cast<int64_t>(i) * a.cols + j;
  float x[32][4];
  if (i0 + 128 <= a.rows && j0 + 128 <= a.cols) {
    load_tile<D, true, NT>(a.X[b], at, a.cols, 32, 4, x);
  } else {
    load_tile<D, false, NT>(a.X[b], at, a.cols, a.rows - i, a.cols - j, x);
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    float top = 0.0f;
#pragma unroll
    for (int e = 0; e < 32; e += 2) top = top3(x[e][c], x[e + 1][c], top);
    const uint32_t byte = mx4_scale_byte(__float_as_uint(top));
    const float scale = scale_operand(byte);
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float y[8] = {x[8 * q][c],     x[8 * q + 1][c], x[8 * q + 2][c], x[8 * q + 3][c],
                          x[8 * q + 4][c], x[8 * q + 5][c], x[8 * q + 6][c], x[8 * q + 7][c]};
      w[q] = byte == 255u ? 0u : code8(y, scale);
    }
    // column 4 l + c at place 32 c + l, so that the lanes' stores are neighbours
    *reinterpret_cast<uint4*>(col_code + (32 * c + l) * kColPitch + 16 * h) = make_uint4(w[0], w[1], w[2], w[3]);
    col_scale[(32 * c + l) * 4 + h] = static_cast<uint8_t>(byte);
  }
  if constexpr (ROWS) {
#pragma unroll
    for (int e8 = 0; e8 < 32; e8 += 8) {
      uint32_t mine = 0;  // scale byte of row e8 + l % 8 of this lane's block of 32 columns
#pragma unroll
      for (int e = e8; e < e8 + 8; ++e) {
        uint32_t top = __float_as_uint(top3(top3(x[e][0], x[e][1], x[e][2]), x[e][3], 0.0f));
        top = dpp_max<kXor1>(top);
        top = dpp_max<kXor2>(top);
        top = dpp_max<kHalfMirror>(top);
        const uint32_t byte = mx4_scale_byte(top);
        const float scale = scale_operand(byte);
        uint32_t w = code_pair<1>(code_pair<0>(0, x[e][0], x[e][1], scale), x[e][2], x[e][3], scale);
        w = byte == 255u ? 0u : w;
        *reinterpret_cast<uint16_t*>(row_code + (32 * h + e) * 64 + 2 * l) = static_cast<uint16_t>(w);
        mine = (l & 7) == e - e8 ? byte : mine;
      }
      row_scale[(32 * h + e8 + (l & 7)) * 4 + (l >> 3)] = static_cast<uint8_t>(mine);
    }
  }
  __syncthreads();
  {
    const int cols_left = a.cols - j0;
    const int64_t line = static_cast<int64_t>(blockIdx.y) * a.cols + j0;
    uint4* codes = static_cast<uint4*>(a.codes_t[b]) + line * 4;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int p = q * kTileThreads + tid, col = p >> 2;
      if (col < cols_left)
        codes[p] = *reinterpret_cast<const uint4*>(col_code + (32 * (col & 3) + (col >> 2)) * kColPitch + 16 * (p & 3));
    }
    if (tid < cols_left)
      static_cast<uint32_t*>(a.scales_t[b])[line + tid] =
          reinterpret_cast<const uint32_t*>(col_scale)[32 * (tid & 3) + (tid >> 2)];
  }
  if constexpr (ROWS) {
    const int rows_left = a.rows - i0;
    const int64_t line = static_cast<int64_t>(blockIdx.x) * a.rows + i0;
    uint4* codes = static_cast<uint4*>(a.codes[b]) + line * 4;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int p = q * kTileThreads + tid;
      if ((p >> 2) < rows_left) codes[p] = reinterpret_cast<const uint4*>(row_code)[p];
    }
    if (tid < rows_left)
      static_cast<uint32_t*>(a.scales[b])[line + tid] = reinterpret_cast<const uint32_t*>(row_scale)[tid];
  }
}

// Values of the code, row-major.  NT: stores past the caches.
template <int D, bool NT>
__global__ __launch_bounds__(kThreads) void mx4_values_kernel(Mx4DequantArgs a, int units) {
  typedef Span<D> V;
  const int b = blockIdx.z, o = threadIdx.x % V::kLanes;
  const int r = blockIdx.x * V::kRows + static_cast<int>(threadIdx.x) / V::kLanes;
  if (r >= a.rows) return;
  const int u0 = blockIdx.y * kUnitsPerThread;
  const uint8_t* codes = static_cast<const uint8_t*>(a.codes[b]);
  const uint8_t* scales = static_cast<const uint8_t*>(a.scales[b]);
  uint32_t code[kUnitsPerThread], byte[kUnitsPerThread];
#pragma unroll
  for (int k = 0; k < kUnitsPerThread; ++k) {
    const int u = u0 + k < units ? u0 + k : units - 1;
    const int64_t line = static_cast<int64_t>(u) * a.rows + r;
    const uint8_t* c = codes + line * 64 + o * (V::kElems / 2);
    code[k] = D == kF32 ? *reinterpret_cast<const uint16_t*>(c) : *reinterpret_cast<const uint32_t*>(c);
    byte[k] = scales[line * 4 + o * V::kElems / kMxBlock];
  }
#pragma unroll
  for (int k = 0; k < kUnitsPerThread; ++k) {
    const int c = (u0 + k) * kMxUnit + V::kElems * o, left = a.cols - c;
    const float s = e8m0_to_f32(byte[k]);
    float y[8];
    const auto p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[k], 1.0f, 0);
    const auto p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[k], 1.0f, 1);
    y[0] = p0[0] * s; y[1] = p0[1] * s; y[2] = p1[0] * s; y[3] = p1[1] * s;
    if constexpr (D != kF32) {
      const auto p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[k], 1.0f, 2);
      const auto p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[k], 1.0f, 3);
      y[4] = p2[0] * s; y[5] = p2[1] * s; y[6] = p3[0] * s; y[7] = p3[1] * s;
    }
    char* const p = static_cast<char*>(a.Y[b]) + (static_cast<int64_t>(r) * a.cols + c) * (D == kF32 ? 4 : 2);
    if (left >= V::kElems) {
      if constexpr (D == kF32) {
        STORE_VEC(reinterpret_cast<u32x4_a4*>(p), __builtin_bit_cast(u32x4_t, make_float4(y[0], y[1], y[2], y[3])));
      } else {
        STORE_VEC(reinterpret_cast<u32x4_a2*>(p),
                  ((u32x4_t){f32x2_to_bf16x2(y[0], y[1]), f32x2_to_bf16x2(y[2], y[3]), f32x2_to_bf16x2(y[4], y[5]),
                             f32x2_to_bf16x2(y[6], y[7])}));
      }
    } else {
#pragma unroll
      for (int e = 0; e < V::kElems; ++e)
        if (e < left) store_from_f32(p, e, D, y[e]);
    }
  }
}

dim3 row_grid(int rows, int per_block, int units, int batch) {
  return dim3((rows + per_block - 1) / per_block, (units + kUnitsPerThread - 1) / kUnitsPerThread, batch);
}

template <int D, bool NT>
void quantize(const Mx4QuantArgs& a, int batch, hipStream_t s) {
  if (a.codes_t[0] == nullptr) {
    const int units = static_cast<int>(mx4_units(a.cols));
    hipLaunchKernelGGL((mx4_rows_kernel<D, NT>), row_grid(a.rows, Span<D>::kRows, units, batch), dim3(kThreads), 0, s, a,
                       units);
    return;
  }
  const dim3 grid(static_cast<uint32_t>(mx4_units(a.cols)), static_cast<uint32_t>(mx4_units(a.rows)), batch);
  if (a.codes[0] != nullptr) {
    hipLaunchKernelGGL((mx4_tile_kernel<D, true, NT>), grid, dim3(kTileThreads), 0, s, a);
  } else {
    hipLaunchKernelGGL((mx4_tile_kernel<D, false, NT>), grid, dim3(kTileThreads), 0, s, a);
  }
}

// Inputs larger than the 256 MB cache are read past it: 3 x 3584x18944 fp32 both
// ways 204 -> 174 us, bf16 120 -> 103; 8192x3584 bf16, still cached, 17 -> 20 us.
constexpr double kStreamBytes = 256.0 * (1 << 20);

template <int D>
void quantize(const Mx4QuantArgs& a, int batch, hipStream_t s) {
  const double bytes = static_cast<double>(a.rows) * a.cols * batch * (D == kF32 ? 4 : 2);
  if (bytes > kStreamBytes) {
    quantize<D, true>(a, batch, s);
  } else {
    quantize<D, false>(a, batch, s);
  }
}

// Whether every row of every matrix starts at a multiple of 64 bytes.  Stores past
// the caches to other rows write the lines that two waves share twice: values of 3
// x 3232x6894 fp32 90 us, through the caches 72, bf16 58 and 30; with 6912 columns,
// all at such places, 51 and 65, 27.1 and 27.7.
bool whole_lines(void* const* ptr, int batch, int cols, int size) {
  uintptr_t bits = static_cast<uintptr_t>(cols) * size;
  for (int i = 0; i < batch; ++i) bits |= reinterpret_cast<uintptr_t>(ptr[i]);
  return (bits & 63u) == 0;
}

// Values pass the caches by at any size: they are four or eight times the codes
// (3 x 3584x18944 fp32: 190 -> 155 us; 4096x4096 fp32 13.8 -> 13.0).
template <int D>
void dequantize(const Mx4DequantArgs& a, int batch, hipStream_t s) {
  const int units = static_cast<int>(mx4_units(a.cols));
  const dim3 grid = row_grid(a.rows, Span<D>::kRows, units, batch), block(kThreads);
  if (whole_lines(a.Y, batch, a.cols, D == kF32 ? 4 : 2)) {
    hipLaunchKernelGGL((mx4_values_kernel<D, true>), grid, block, 0, s, a, units);
  } else {
    hipLaunchKernelGGL((mx4_values_kernel<D, false>), grid, block, 0, s, a, units);
  }
}

}  // namespace

hipError_t launch_mx4_quantize(const Mx4QuantArgs& a, int batch, hipStream_t s) {
  switch (a.x_dtype) {
    case kF32: quantize<kF32>(a, batch, s); break;
    case kBF16: quantize<kBF16>(a, batch, s); break;
    default: quantize<kF16>(a, batch, s); break;
  }
  return hipGetLastError();
}

hipError_t launch_mx4_dequantize(const Mx4DequantArgs& a, int batch, hipStream_t s) {
  if (a.y_dtype == kF32) {
    dequantize<kF32>(a, batch, s);
  } else {
    dequantize<kBF16>(a, batch, s);
  }
  return hipGetLastError();
}

}  // namespace muon

using namespace muon;

namespace {

bool mx4_shape_ok(int batch, int rows, int cols) {
  return batch >= 1 && rows >= 1 && cols >= 1 && rows <= MUON_MAX_DIM && cols <= MUON_MAX_DIM;
}

// A host array of `batch` non-null device pointers, multiples of `align`.
bool pointers_ok(int batch, const void* const* p, uintptr_t align = 1) {
  if (p == nullptr) return false;
  for (int i = 0; i < batch; ++i)
    if (p[i] == nullptr || (reinterpret_cast<uintptr_t>(p[i]) & (align - 1)) != 0) return false;
  return true;
}
constexpr uintptr_t kCodeAlign = 16, kScaleAlign = 4;

template <class T>
void take(T* to, T const* from, int at, int count) {
  for (int i = 0; i < count; ++i) to[i] = from != nullptr ? from[at + i] : nullptr;
}

bool mx4_type_ok(muon_dtype d) { return d == MUON_F32 || d == MUON_BF16 || d == MUON_F16; }

double code_bytes(double rows, double k) { return rows * static_cast<double>(mx4_units(static_cast<int64_t>(k))) * 68.0; }

// One matrix's codes are addressed with 32-bit byte offsets in the product.
bool operand_ok(int rows, int k) { return mx4_units(k) * rows * 64 < (static_cast<int64_t>(1) << 31); }

}  // namespace

extern "C" {

muon_status muon_mx4_quantize(int batch, int rows, int cols, const void* const* X, muon_dtype x_dtype,
                              void* const* codes, void* const* scales, void* const* codes_t, void* const* scales_t,
                              void* stream) {
  if (!mx4_shape_ok(batch, rows, cols) || !mx4_type_ok(x_dtype)) return MUON_ERR_INVALID_ARG;
  if ((codes == nullptr) != (scales == nullptr) || (codes_t == nullptr) != (scales_t == nullptr))
    return MUON_ERR_INVALID_ARG;
  if (codes == nullptr && codes_t == nullptr) return MUON_ERR_INVALID_ARG;
  const void* const* arrays[5] = {X, codes, scales, codes_t, scales_t};
  const uintptr_t align[5] = {1, kCodeAlign, kScaleAlign, kCodeAlign, kScaleAlign};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < i; ++j)
      if (arrays[i] != nullptr && arrays[i] == arrays[j]) return MUON_ERR_INVALID_ARG;
    if ((i == 0 || arrays[i] != nullptr) && !pointers_ok(batch, arrays[i], align[i])) return MUON_ERR_INVALID_ARG;
  }
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const double r = rows, c = cols;
  const double bytes = r * c * (x_dtype == MUON_F32 ? 4.0 : 2.0) + (codes != nullptr ? code_bytes(r, c) : 0.0) +
                       (codes_t != nullptr ? code_bytes(c, r) : 0.0);
  for (int at = 0; at < batch; at += kMxBatch) {
    const int count = batch - at < kMxBatch ? batch - at : kMxBatch;
    Mx4QuantArgs a;
    a.x_dtype = x_dtype;
    a.rows = rows;
    a.cols = cols;
    take(a.X, X, at, count);
    take(a.codes, codes, at, count);
    take(a.scales, scales, at, count);
    take(a.codes_t, codes_t, at, count);
    take(a.scales_t, scales_t, at, count);
    if (traced_launch(s, codes_t != nullptr ? "mx4_tile_kernel" : "mx4_rows_kernel", "mx4_quantize", 0.0, bytes * count,
                      [&] { return launch_mx4_quantize(a, count, s); }) != hipSuccess)
      return MUON_ERR_HIP;
  }
  return MUON_OK;
}

muon_status muon_mx4_dequantize(int batch, int rows, int cols, const void* const* codes, const void* const* scales,
                                void* const* Y, muon_dtype y_dtype, void* stream) {
  if (!mx4_shape_ok(batch, rows, cols) || !pointers_ok(batch, codes, kCodeAlign) ||
      !pointers_ok(batch, scales, kScaleAlign) || !pointers_ok(batch, Y))
    return MUON_ERR_INVALID_ARG;
  if (!mx4_type_ok(y_dtype) || codes == scales || static_cast<const void*>(codes) == Y ||
      static_cast<const void*>(scales) == Y)
    return MUON_ERR_INVALID_ARG;
  if (y_dtype == MUON_F16) return MUON_ERR_UNSUPPORTED;  // the code's range is that of binary32
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const double bytes = static_cast<double>(rows) * cols * (y_dtype == MUON_F32 ? 4.0 : 2.0) + code_bytes(rows, cols);
  for (int at = 0; at < batch; at += kMxBatch) {
    const int count = batch - at < kMxBatch ? batch - at : kMxBatch;
    Mx4DequantArgs a;
    a.rows = rows;
    a.cols = cols;
    a.y_dtype = y_dtype;
    take(a.codes, codes, at, count);
    take(a.scales, scales, at, count);
    take(a.Y, Y, at, count);
    if (traced_launch(s, "mx4_values_kernel", "mx4_dequantize", 0.0, bytes * count,
                      [&] { return launch_mx4_dequantize(a, count, s); }) != hipSuccess)
      return MUON_ERR_HIP;
  }
  return MUON_OK;
}

size_t muon_mx4_workspace_size(int batch, int m, int n, int k) {
  if (!mx4_shape_ok(batch, m, k) || !mx4_shape_ok(batch, n, k) || !operand_ok(m, k) || !operand_ok(n, k)) return 0;
  // one launch at a time uses it: the largest need is that of a whole launch or of the last one
  const int whole = batch < kMxBatch ? batch : kMxBatch, rest = batch % kMxBatch;
  size_t bytes = mx4_plan(whole, m, n, k).bytes;
  if (rest > 0) {
    const size_t last = mx4_plan(rest, m, n, k).bytes;
    bytes = last > bytes ? last : bytes;
  }
  return bytes > 256 ? (bytes + 255) / 256 * 256 : 256;
}

muon_status muon_mx4_matmul(int batch, int m, int n, int k, const void* const* A_codes, const void* const* A_scales,
                            const void* const* B_codes, const void* const* B_scales, void* const* C,
                            muon_dtype c_dtype, int accumulate, void* workspace, size_t ws_bytes, void* stream) {
  const size_t need = muon_mx4_workspace_size(batch, m, n, k);
  if (need == 0) return MUON_ERR_INVALID_ARG;
  const void* const* in[4] = {A_codes, A_scales, B_codes, B_scales};
  if (!pointers_ok(batch, C)) return MUON_ERR_INVALID_ARG;
  for (int i = 0; i < 4; ++i)  // A and B may be one matrix (A A^T); C is written
    if (!pointers_ok(batch, in[i], i % 2 == 0 ? kCodeAlign : kScaleAlign) || static_cast<const void*>(in[i]) == C)
      return MUON_ERR_INVALID_ARG;
  if (!mx4_type_ok(c_dtype) || (accumulate != 0 && accumulate != 1)) return MUON_ERR_INVALID_ARG;
  if (c_dtype == MUON_F16) return MUON_ERR_UNSUPPORTED;
  if (workspace == nullptr || ws_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return MUON_ERR_WORKSPACE;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const double mn = static_cast<double>(m) * n;
  const double bytes = code_bytes(m, k) + code_bytes(n, k) +
                       mn * (c_dtype == MUON_F32 ? 4.0 : 2.0) * (accumulate ? 2.0 : 1.0);
  for (int at = 0; at < batch; at += kMxBatch) {
    const int count = batch - at < kMxBatch ? batch - at : kMxBatch;
    const Mx4Plan plan = mx4_plan(count, m, n, k);
    Mx4GemmArgs a;
    a.batch = count;
    a.m = m;
    a.n = n;
    a.k = k;
    a.units = static_cast<int>(mx4_units(k));
    a.c_dtype = c_dtype;
    a.accumulate = accumulate;
    a.pieces = plan.pieces;
    a.piece_units = plan.piece_units;
    a.partial = static_cast<float*>(workspace);
    take(a.A, A_codes, at, count);
    take(a.As, A_scales, at, count);
    take(a.B, B_codes, at, count);
    take(a.Bs, B_scales, at, count);
    take(a.C, C, at, count);
    const char* kernel = plan.kind == kMxFewRows ? "mx4_few_rows_kernel" : "mx4_tile_gemm_kernel";
    if (traced_launch(s, kernel, "mx4_matmul", 2.0 * count * mn * k, bytes * count,
                      [&] { return launch_mx4_gemm(a, plan.kind, s); }) != hipSuccess)
      return MUON_ERR_HIP;
    if (plan.pieces > 1 &&
        traced_launch(s, "mx4_join_kernel", "mx4_join", 0.0, count * mn * (4.0 * plan.pieces + (c_dtype == MUON_F32 ? 4.0 : 2.0)),
                      [&] { return launch_mx4_join(a, s); }) != hipSuccess)
      return MUON_ERR_HIP;
  }
  return MUON_OK;
}

}  // extern "C"

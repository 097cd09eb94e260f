// The 8-bit code with a scale for each block of 128: 128 consecutive elements of a
// row, or a tile of 128 x 128, share a power of two (one E8M0 byte); each element is
// an e4m3 or e5m2 float.  The scale is the smallest power of two with which the
// block's largest magnitude is in the format's range, elements are rounded to
// nearest even.  Both steps are exact in fp32, so the code of a matrix does not
// depend on how it is computed.
#include "../../include/muon.h"
#include "muon_convert.h"
#include "muon_fp8.h"
#include "muon_internal.h"

namespace muon {
namespace {

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef short i16x2_t __attribute__((ext_vector_type(2)));

// Rows of odd length start anywhere: loads and stores of 8 and 16 bytes that need
// the alignment of one element only.
typedef u32x2_t u32x2_a2 __attribute__((aligned(2)));
typedef u32x4_t u32x4_a2 __attribute__((aligned(2)));
typedef u32x4_t u32x4_a4 __attribute__((aligned(4)));

template <int D>
__device__ __forceinline__ float half_of(uint32_t w, int upper) {
  const uint16_t h = static_cast<uint16_t>(upper ? w >> 16 : w);
  return D == kBF16 ? bf16_to_f32(h) : f16_to_f32(h);
}

// (Macro: a template parameter would drop the pointer type's alignment.)
#define LOAD_VEC(p) (NT ? __builtin_nontemporal_load(p) : *(p))

// Scale as the converters take it: its exponent field is the scale byte.
__device__ __forceinline__ float scale_operand(uint32_t byte) { return __uint_as_float(byte << 23); }

// Four codes of x / scale (nearest even) as one word, 0 where the scale is NaN.
template <int F>
__device__ __forceinline__ uint32_t code4(float x0, float x1, float x2, float x3, uint32_t byte) {
  const float scale = scale_operand(byte);
  i16x2_t w = {0, 0};
  if constexpr (F == kE4M3) {
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, x0, x1, scale, false);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, x2, x3, scale, true);
  } else {
    w = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(w, x0, x1, scale, false);
    w = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(w, x2, x3, scale, true);
  }
  return byte == 255u ? 0u : __builtin_bit_cast(uint32_t, w);
}

// Largest magnitude of three, NaN if one is NaN.
__device__ __forceinline__ float top3(float a, float b, float c) {
  return __builtin_elementwise_maximum(__builtin_elementwise_maximum(fabsf(a), fabsf(b)), fabsf(c));
}

__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x) {  // of non-negative floats' bits (NaN is largest)
  return larger(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), CTRL, 0xf, 0xf, true)));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;  // quads, reversal within 8 and 16 lanes
__device__ __forceinline__ uint32_t max16(uint32_t x) {                          // over 16 neighbouring lanes
  return dpp_max<kMirror>(dpp_max<kHalfMirror>(dpp_max<kXor2>(dpp_max<kXor1>(x))));
}

// ---------------------------------------------------------------------------
// Rows of X to or from rows of units: 16 threads take a unit of a row, each 8
// elements (16-bit types: 16 bytes in a row; fp32: 16 bytes of either piece), so that
// a wave's access is four or eight whole runs of 256 bytes, for kUnitsPerThread
// units one after the other with all loads out first.  Bound by memory: 3 x 3584 x
// 18944 fp32 165 us, 6.2 TB/s.
// ---------------------------------------------------------------------------
constexpr int kThreads = 256;
constexpr int kUnitsPerThread = 4;
constexpr int kRows = kThreads / 16;  // of a block

template <int D>
__device__ __forceinline__ int column(int o, int e) {  // of element e of thread o in its unit
  return D == kF32 ? 64 * (e >> 2) + 4 * o + (e & 3) : 8 * o + e;
}

template <int D, bool NT>
__device__ __forceinline__ void load_span(const void* X, int64_t at, int o, int left, uint32_t (&r)[8]) {
  if constexpr (D == kF32) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = column<D>(o, 4 * h);
      const uint32_t* p = static_cast<const uint32_t*>(X) + at + c;
      if (c + 4 <= left) {
        const u32x4_t v = LOAD_VEC(reinterpret_cast<const u32x4_a4*>(p));
#pragma unroll
        for (int e = 0; e < 4; ++e) r[4 * h + e] = v[e];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) r[4 * h + e] = c + e < left ? p[e] : 0u;
      }
    }
  } else {
    const int c = column<D>(o, 0);
    const uint16_t* p = static_cast<const uint16_t*>(X) + at + c;
    if (c + 8 <= left) {
      const u32x4_t v = LOAD_VEC(reinterpret_cast<const u32x4_a2*>(p));
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] = v[e];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        r[e] = (c + 2 * e < left ? p[2 * e] : 0u) | (c + 2 * e + 1 < left ? static_cast<uint32_t>(p[2 * e + 1]) << 16 : 0u);
    }
  }
}

template <int D, int F, bool NT>
__global__ __launch_bounds__(kThreads) void fp8_rows_kernel(Fp8QuantArgs a, int units) {
  const int b = blockIdx.z, o = threadIdx.x & 15, r = blockIdx.x * kRows + (threadIdx.x >> 4);
  if (r >= a.rows) return;  // all threads of a row together
  const int u0 = blockIdx.y * kUnitsPerThread;
  const int64_t pitch = fp8_pitch(a.rows);
  uint8_t* codes = static_cast<uint8_t*>(a.codes[b]);
  uint8_t* scales = static_cast<uint8_t*>(a.scales[b]);
  uint32_t raw[kUnitsPerThread][8];
#pragma unroll
  for (int k = 0; k < kUnitsPerThread; ++k) {
    const int c = (u0 + k) * kF8Unit;
    load_span<D, NT>(a.X[b], static_cast<int64_t>(r) * a.cols + c, o, a.cols - c, raw[k]);
  }
#pragma unroll
  for (int k = 0; k < kUnitsPerThread; ++k) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = D == kF32 ? __uint_as_float(raw[k][e]) : half_of<D>(raw[k][e >> 1], e & 1);
    const uint32_t top =
        max16(__float_as_uint(top3(top3(x[0], x[1], x[2]), top3(x[3], x[4], x[5]), top3(x[6], x[7], 0.0f))));
    const uint32_t byte = fp8_scale_byte<F>(top);
    const uint32_t lo = code4<F>(x[0], x[1], x[2], x[3], byte), hi = code4<F>(x[4], x[5], x[6], x[7], byte);
    const int u = u0 + k;
    if (u < units) {
      uint8_t* const c = codes + (static_cast<int64_t>(2 * u) * a.rows + r) * kF8Piece;
      const int64_t piece = static_cast<int64_t>(a.rows) * kF8Piece;
      if constexpr (D == kF32) {
        *reinterpret_cast<uint32_t*>(c + 4 * o) = lo;
        *reinterpret_cast<uint32_t*>(c + piece + 4 * o) = hi;
      } else {
        *reinterpret_cast<uint2*>(c + (o >> 3) * piece + 8 * (o & 7)) = make_uint2(lo, hi);
      }
      if (o == 0) scales[u * pitch + r] = static_cast<uint8_t>(byte);
    }
  }
}

// ---------------------------------------------------------------------------
// Codes along columns, along both, or of tiles, from one read of X: a block of 256
// threads takes a 128 x 128 tile, a thread 16 rows x 4 columns of it in registers.
// The largest magnitudes of its columns and rows (or of the whole tile) meet in LDS;
// the codes are put together there too, and written in whole lines: each
// orientation's are two contiguous runs of 8 KB.  With row counts a tile starts at
// its group's first row, and what is behind the group's last is zero.  Bound by memory:
// 3 x 3584 x 18944 fp32 in tiles, both ways, 207 us, 5.9 TB/s; small calls by the launch (5 x
// 3584 bf16 with its values, two launches, 11.4 us).
// ---------------------------------------------------------------------------
constexpr int kTileRows = 16;
constexpr int kCodePitch = 144;  // bytes of a row's or column's codes in LDS: 128, and 16 against bank conflicts

// The 16 x 4 elements of a thread; rows_left and cols_left of the matrix are there,
// from row 0 and column 0 of them on (none if 0 or less), the others read as zero.
// `at` is the first element's place.  Where not all are there, the rows behind the
// end read the last one, and the columns over the end the row's last four, shifted
// into place, so that these tiles too have all their loads out at once.
template <int D, bool FULL, bool NT>
__device__ __forceinline__ void load_tile(const void* X, int64_t at, int64_t pitch, int rows_left, int cols_left,
                                          float (&x)[kTileRows][4]) {
  if (FULL || pitch >= 4) {
    const int over = FULL || cols_left >= 4 ? 0 : 4 - cols_left;  // columns of the four that are not there
    const int last = rows_left - 1;
    const int64_t from = at - over;
    if constexpr (D == kF32) {
      u32x4_t v[kTileRows];
#pragma unroll
      for (int e = 0; e < kTileRows; ++e)
        v[e] = LOAD_VEC(reinterpret_cast<const u32x4_a4*>(static_cast<const float*>(X) + from +
                                                         (FULL || e < last ? e : last) * pitch));
#pragma unroll
      for (int e = 0; e < kTileRows; ++e) {
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
      u32x2_t v[kTileRows];
#pragma unroll
      for (int e = 0; e < kTileRows; ++e)
        v[e] = LOAD_VEC(reinterpret_cast<const u32x2_a2*>(static_cast<const uint16_t*>(X) + from +
                                                         (FULL || e < last ? e : last) * pitch));
#pragma unroll
      for (int e = 0; e < kTileRows; ++e) {
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
    for (int e = 0; e < kTileRows; ++e)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        x[e][c] = e < rows_left && c < cols_left ? load_as_f32(X, at + e * pitch + c, D) : 0.0f;
  }
}

template <int D, int F, bool NT, bool PAST>
__global__ __launch_bounds__(kThreads) void fp8_tile_kernel(Fp8QuantArgs a) {
  __shared__ __align__(16) uint8_t col_code[128 * kCodePitch];
  __shared__ __align__(16) uint8_t row_code[128 * kCodePitch];
  __shared__ __align__(16) uint32_t col_top[8][128];
  __shared__ __align__(16) uint8_t col_scale[128], row_scale[128];
  __shared__ uint32_t wave_top[4];
  const int b = blockIdx.z, tid = threadIdx.x, h = tid >> 5, l = tid & 31, wave = tid >> 6;
  const bool rows = a.codes[b] != nullptr, tile = a.tile != 0;
  bool cols = a.codes_t[b] != nullptr;
  int i0 = blockIdx.y * 128, end = a.rows, unit = blockIdx.y;  // first row, end of its group, unit of the columns' code
  if (a.counts != nullptr) {
    const auto count = [&](int g) { return group_count(a.counts, g, a.groups, a.rows); };
    const RowTiles<128, decltype(count)> tiles{count, a.rows, a.groups + (rows ? 1 : 0), 0};
    const RowTile t = tiles.of(blockIdx.y, 1, tid & 63);
    if (t.group < 0) return;
    i0 = t.begin + t.tile * 128;
    end = t.end;
    unit = t.before + t.tile;
    cols = cols && t.group < a.groups;  // rows behind the last group are in no column's code
  }
  const int j0 = blockIdx.x * 128;
  const int i = i0 + kTileRows * h, j = j0 + 4 * l;
  const int64_t at = static_cast<int64_t>(i) * a.cols + j;
  float x[kTileRows][4];
  if (i0 + 128 <= end && j0 + 128 <= a.cols) {
    load_tile<D, true, NT>(a.X[b], at, a.cols, kTileRows, 4, x);
  } else {
    load_tile<D, false, NT>(a.X[b], at, a.cols, end - i, a.cols - j, x);
  }
  uint32_t col_byte[4], row_bytes[4];  // of this thread's columns; of its rows, four in a word
  if (tile) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < kTileRows; ++e)
      top = larger(top, __float_as_uint(top3(top3(x[e][0], x[e][1], x[e][2]), x[e][3], 0.0f)));
    top = max16(top);
    top = larger(top, __shfl_xor(top, 16));
    top = larger(top, __shfl_xor(top, 32));
    if ((tid & 63) == 0) wave_top[wave] = top;
    __syncthreads();
    const uint32_t byte = fp8_scale_byte<F>(larger(larger(wave_top[0], wave_top[1]), larger(wave_top[2], wave_top[3])));
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      col_byte[c] = byte;
      row_bytes[c] = byte * 0x01010101u;
    }
    if (tid < 128) {
      col_scale[tid] = static_cast<uint8_t>(byte);
      row_scale[tid] = static_cast<uint8_t>(byte);
    }
  } else {
    if (cols) {
      uint4 top;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float t = 0.0f;
#pragma unroll
        for (int e = 0; e < kTileRows; e += 2) t = top3(x[e][c], x[e + 1][c], t);
        (&top.x)[c] = __float_as_uint(t);
      }
      *reinterpret_cast<uint4*>(&col_top[h][4 * l]) = top;
    }
    if (rows) {
      uint32_t mine = 0;  // largest magnitude of row l % 16 in this thread's 16 lanes
#pragma unroll
      for (int e = 0; e < kTileRows; ++e) {
        const uint32_t top = max16(__float_as_uint(top3(top3(x[e][0], x[e][1], x[e][2]), x[e][3], 0.0f)));
        mine = (l & 15) == e ? top : mine;
      }
      mine = larger(mine, __shfl_xor(mine, 16));
      if (l < 16) row_scale[kTileRows * h + l] = static_cast<uint8_t>(fp8_scale_byte<F>(mine));
    }
    __syncthreads();
    if (cols) {
      uint4 top = *reinterpret_cast<const uint4*>(&col_top[0][4 * l]);
#pragma unroll
      for (int q = 1; q < 8; ++q) {
        const uint4 t = *reinterpret_cast<const uint4*>(&col_top[q][4 * l]);
        top = make_uint4(larger(top.x, t.x), larger(top.y, t.y), larger(top.z, t.z), larger(top.w, t.w));
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) col_byte[c] = fp8_scale_byte<F>((&top.x)[c]);
      if (h == 0)
        *reinterpret_cast<uint32_t*>(col_scale + 4 * l) =
            col_byte[0] | (col_byte[1] << 8) | (col_byte[2] << 16) | (col_byte[3] << 24);
    }
    const uint4 t = *reinterpret_cast<const uint4*>(row_scale + kTileRows * h);
    row_bytes[0] = t.x; row_bytes[1] = t.y; row_bytes[2] = t.z; row_bytes[3] = t.w;
  }
  if (cols) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) w[q] = code4<F>(x[4 * q][c], x[4 * q + 1][c], x[4 * q + 2][c], x[4 * q + 3][c], col_byte[c]);
      // column 4 l + c at place 32 c + l, so that the lanes' stores are neighbours
      *reinterpret_cast<uint4*>(col_code + (32 * c + l) * kCodePitch + kTileRows * h) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  if (rows) {
#pragma unroll
    for (int e = 0; e < kTileRows; ++e)
      *reinterpret_cast<uint32_t*>(row_code + (kTileRows * h + e) * kCodePitch + 4 * l) =
          code4<F>(x[e][0], x[e][1], x[e][2], x[e][3], (row_bytes[e >> 2] >> (8 * (e & 3))) & 255u);
  }
  __syncthreads();
  const auto put = [&](u32x4_t* to, const uint8_t* from) {
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(from);
    if constexpr (PAST) {
      __builtin_nontemporal_store(v, to);
    } else {
      *to = v;
    }
  };
  if (cols) {
    const int left = a.cols - j0;
    u32x4_t* codes = static_cast<u32x4_t*>(a.codes_t[b]);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int p = q * kThreads + tid, half = p >> 9, col = (p >> 2) & 127, chunk = p & 3;
      if (col < left)
        put(codes + (static_cast<int64_t>(2 * unit + half) * a.cols + j0 + col) * 4 + chunk,
            col_code + (32 * (col & 3) + (col >> 2)) * kCodePitch + half * kF8Piece + chunk * 16);
    }
    if (tid < 128 && tid < left)
      static_cast<uint8_t*>(a.scales_t[b])[unit * fp8_pitch(a.cols) + j0 + tid] = col_scale[tid];
  }
  if (rows) {
    const int left = end - i0;
    u32x4_t* codes = static_cast<u32x4_t*>(a.codes[b]);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int p = q * kThreads + tid, half = p >> 9, row = (p >> 2) & 127, chunk = p & 3;
      if (row < left)
        put(codes + (static_cast<int64_t>(2 * blockIdx.x + half) * a.rows + i0 + row) * 4 + chunk,
            row_code + row * kCodePitch + half * kF8Piece + chunk * 16);
    }
    if (tid < 128 && tid < left)
      static_cast<uint8_t*>(a.scales[b])[blockIdx.x * fp8_pitch(a.rows) + i0 + tid] = row_scale[tid];
  }
}

// Values of the code, row-major: 16 threads take a unit of a row as in the rows'
// code.  NT: stores past the caches.  3 x 3584 x 18944 fp32 151 us, 6.7 TB/s.
template <int D, int F, bool NT>
__global__ __launch_bounds__(kThreads) void fp8_values_kernel(Fp8DequantArgs a, int units) {
  const int b = blockIdx.z, o = threadIdx.x & 15, r = blockIdx.x * kRows + (threadIdx.x >> 4);
  if (r >= a.rows) return;
  const int u0 = blockIdx.y * kUnitsPerThread;
  const int64_t pitch = fp8_pitch(a.rows), piece = static_cast<int64_t>(a.rows) * kF8Piece;
  const uint8_t* codes = static_cast<const uint8_t*>(a.codes[b]) + static_cast<int64_t>(r) * kF8Piece;
  const uint8_t* scales = static_cast<const uint8_t*>(a.scales[b]) + r;
  uint32_t word[kUnitsPerThread][2], byte[kUnitsPerThread];
#pragma unroll
  for (int k = 0; k < kUnitsPerThread; ++k) {
    const int u = u0 + k < units ? u0 + k : units - 1;
    const uint8_t* c = codes + 2 * u * piece;
    if constexpr (D == kF32) {
      word[k][0] = *reinterpret_cast<const uint32_t*>(c + 4 * o);
      word[k][1] = *reinterpret_cast<const uint32_t*>(c + piece + 4 * o);
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(c + (o >> 3) * piece + 8 * (o & 7));
      word[k][0] = w.x;
      word[k][1] = w.y;
    }
    byte[k] = scales[u * pitch];
  }
#pragma unroll
  for (int k = 0; k < kUnitsPerThread; ++k) {
    const float s = fp8_scale_value(byte[k]);
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const bool upper = (e & 2) != 0;
      f32x2_t p;
      if constexpr (F == kE4M3) {
        p = upper ? __builtin_bit_cast(f32x2_t, __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(word[k][e >> 2], 1.0f, true))
                  : __builtin_bit_cast(f32x2_t, __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(word[k][e >> 2], 1.0f, false));
      } else {
        p = upper ? __builtin_bit_cast(f32x2_t, __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(word[k][e >> 2], 1.0f, true))
                  : __builtin_bit_cast(f32x2_t, __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(word[k][e >> 2], 1.0f, false));
      }
      y[e] = p[0] * s;
      y[e + 1] = p[1] * s;
    }
    const int c0 = (u0 + k) * kF8Unit, left = a.cols - c0;
    constexpr int kSize = D == kF32 ? 4 : 2, kRun = D == kF32 ? 4 : 8;
    char* const p = static_cast<char*>(a.Y[b]) + (static_cast<int64_t>(r) * a.cols + c0) * kSize;
#pragma unroll
    for (int g = 0; g < 8; g += kRun) {
      const int c = column<D>(o, g);
      char* const q = p + c * kSize;
      if (c + kRun <= left) {
        u32x4_t v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = D == kF32 ? __float_as_uint(y[(g + e) & 7]) : f32x2_to_bf16x2(y[(2 * e) & 7], y[(2 * e + 1) & 7]);
        if constexpr (NT) {
          if constexpr (D == kF32) {
            __builtin_nontemporal_store(v, reinterpret_cast<u32x4_a4*>(q));
          } else {
            __builtin_nontemporal_store(v, reinterpret_cast<u32x4_a2*>(q));
          }
        } else {
          if constexpr (D == kF32) {
            *reinterpret_cast<u32x4_a4*>(q) = v;
          } else {
            *reinterpret_cast<u32x4_a2*>(q) = v;
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < kRun; ++e)
          if (c + e < left) store_from_f32(q, e, D, y[g + e]);
      }
    }
  }
}

template <int D, int F, bool NT, bool PAST>
void quantize(const Fp8QuantArgs& a, int batch, hipStream_t s) {
  const int64_t col_units = fp8_units(a.cols);
  if (a.codes_t[0] == nullptr && a.tile == 0) {
    const dim3 grid((a.rows + kRows - 1) / kRows, static_cast<uint32_t>((col_units + kUnitsPerThread - 1) / kUnitsPerThread),
                    batch);
    hipLaunchKernelGGL((fp8_rows_kernel<D, F, NT>), grid, dim3(kThreads), 0, s, a, static_cast<int>(col_units));
    return;
  }
  const int64_t row_units =
      a.counts == nullptr ? fp8_units(a.rows) : a.rows / kF8Unit + a.groups + (a.codes[0] != nullptr ? 1 : 0);
  const dim3 grid(static_cast<uint32_t>(col_units), static_cast<uint32_t>(row_units), batch);
  hipLaunchKernelGGL((fp8_tile_kernel<D, F, NT, PAST>), grid, dim3(kThreads), 0, s, a);
}

// A call that moves more than the 256 MB cache holds reads past it (us): 16380x7168
// bf16 along rows 66 -> 56, both ways 90 -> 73; 4096x18944 bf16 both ways 56 -> 54,
// along rows, which fits, 35 -> 39.  One of several times that also writes a tile's
// codes past it: 3 x 3584x18944 fp32 both ways 224 -> 206, one of them 65 -> 70.
constexpr double kCacheBytes = 256.0 * (1 << 20), kPastBytes = 3.0 * kCacheBytes;

template <int D, int F>
void quantize(const Fp8QuantArgs& a, int batch, hipStream_t s) {
  const double elements = static_cast<double>(a.rows) * a.cols * batch;
  const double bytes = elements * ((D == kF32 ? 4 : 2) + (a.codes[0] != nullptr ? 1 : 0) + (a.codes_t[0] != nullptr ? 1 : 0));
  if (bytes > kPastBytes) {
    quantize<D, F, true, true>(a, batch, s);
  } else if (bytes > kCacheBytes) {
    quantize<D, F, true, false>(a, batch, s);
  } else {
    quantize<D, F, false, false>(a, batch, s);
  }
}
template <int D>
void quantize(const Fp8QuantArgs& a, int batch, hipStream_t s) {
  if (a.format == kE4M3) {
    quantize<D, kE4M3>(a, batch, s);
  } else {
    quantize<D, kE5M2>(a, batch, s);
  }
}

// Whether every row of every matrix starts at a multiple of 64 bytes: stores past the
// caches to other rows write the lines that two waves share twice.
bool whole_lines(void* const* ptr, int batch, int cols, int size) {
  uintptr_t bits = static_cast<uintptr_t>(cols) * size;
  for (int i = 0; i < batch; ++i) bits |= reinterpret_cast<uintptr_t>(ptr[i]);
  return (bits & 63u) == 0;
}

template <int D, int F>
void dequantize(const Fp8DequantArgs& a, int batch, hipStream_t s) {
  const int units = static_cast<int>(fp8_units(a.cols));
  const dim3 grid((a.rows + kRows - 1) / kRows, (units + kUnitsPerThread - 1) / kUnitsPerThread, batch), block(kThreads);
  if (whole_lines(a.Y, batch, a.cols, D == kF32 ? 4 : 2)) {
    hipLaunchKernelGGL((fp8_values_kernel<D, F, true>), grid, block, 0, s, a, units);
  } else {
    hipLaunchKernelGGL((fp8_values_kernel<D, F, false>), grid, block, 0, s, a, units);
  }
}
template <int D>
void dequantize(const Fp8DequantArgs& a, int batch, hipStream_t s) {
  if (a.format == kE4M3) {
    dequantize<D, kE4M3>(a, batch, s);
  } else {
    dequantize<D, kE5M2>(a, batch, s);
  }
}

}  // namespace

hipError_t launch_fp8_quantize(const Fp8QuantArgs& a, int batch, hipStream_t s) {
  switch (a.x_dtype) {
    case kF32: quantize<kF32>(a, batch, s); break;
    case kBF16: quantize<kBF16>(a, batch, s); break;
    default: quantize<kF16>(a, batch, s); break;
  }
  return hipGetLastError();
}

hipError_t launch_fp8_dequantize(const Fp8DequantArgs& a, int batch, hipStream_t s) {
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

bool shape_ok(int batch, int rows, int cols) {
  return batch >= 1 && rows >= 1 && cols >= 1 && rows <= MUON_MAX_DIM && cols <= MUON_MAX_DIM;
}

bool pointer_ok(const void* p, uintptr_t align) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (align - 1)) == 0; }

// A host array of `batch` non-null device pointers, multiples of `align`.
bool pointers_ok(int batch, const void* const* p, uintptr_t align = 1) {
  if (p == nullptr) return false;
  for (int i = 0; i < batch; ++i)
    if (!pointer_ok(p[i], align)) return false;
  return true;
}
constexpr uintptr_t kAlign = 16;  // of codes and scales

template <class T>
void take(T* to, T const* from, int at, int count) {
  for (int i = 0; i < count; ++i) to[i] = from != nullptr ? from[at + i] : nullptr;
}

bool type_ok(muon_dtype d) { return d == MUON_F32 || d == MUON_BF16 || d == MUON_F16; }
bool format_ok(muon_fp8_format f) { return f == MUON_E4M3 || f == MUON_E5M2; }
double size_of(muon_dtype d) { return d == MUON_F32 ? 4.0 : 2.0; }

double code_bytes(double rows, double units) { return rows * units * (kF8Unit + 1.0); }

// Row counts on the device; rows x (groups + 1) fit 31 bits, so that no sum of counts wraps.
bool groups_ok(const int32_t* counts, int groups, int rows) {
  return pointer_ok(counts, 4) && groups >= 1 && groups <= MUON_MAX_DIM &&
         static_cast<int64_t>(rows) * (groups + 1) < (static_cast<int64_t>(1) << 31);
}

// A launch's blocks fit 31 bits in tiles of 64 x 128, the smallest.
bool grid_ok(int64_t outer, int64_t m, int64_t n) {
  return outer * ((m + 63) / 64) * ((n + 127) / 128) < (static_cast<int64_t>(1) << 31);
}

const char* kernel_name(Fp8Kind kind, const char* few, const char* tiles) { return kind == kF8FewRows ? few : tiles; }

}  // namespace

extern "C" {

muon_status muon_fp8_quantize(int batch, int rows, int cols, const void* const* X, muon_dtype x_dtype, int tile,
                              muon_fp8_format format, const int32_t* counts, int groups, void* const* codes,
                              void* const* scales, void* const* codes_t, void* const* scales_t, void* stream) {
  if (!shape_ok(batch, rows, cols) || !type_ok(x_dtype) || !format_ok(format) || (tile != 0 && tile != 1))
    return MUON_ERR_INVALID_ARG;
  if ((codes == nullptr) != (scales == nullptr) || (codes_t == nullptr) != (scales_t == nullptr))
    return MUON_ERR_INVALID_ARG;
  if (codes == nullptr && codes_t == nullptr) return MUON_ERR_INVALID_ARG;
  if (counts == nullptr ? groups != 0 : (!groups_ok(counts, groups, rows) || batch != 1 || tile != 0 || codes_t == nullptr))
    return MUON_ERR_INVALID_ARG;
  if (counts != nullptr && rows / kF8Unit + groups + 1 > 65535) return MUON_ERR_INVALID_ARG;  // the launch's row tiles
  const void* const* arrays[5] = {X, codes, scales, codes_t, scales_t};
  const uintptr_t align[5] = {1, kAlign, kAlign, kAlign, kAlign};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < i; ++j)
      if (arrays[i] != nullptr && arrays[i] == arrays[j]) return MUON_ERR_INVALID_ARG;
    if ((i == 0 || arrays[i] != nullptr) && !pointers_ok(batch, arrays[i], align[i])) return MUON_ERR_INVALID_ARG;
  }
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const double r = rows, c = cols;
  const double bytes = r * c * size_of(x_dtype) + (codes != nullptr ? code_bytes(r, fp8_units(cols)) : 0.0) +
                       (codes_t != nullptr ? code_bytes(c, fp8_units(rows)) : 0.0);
  for (int at = 0; at < batch; at += kF8Batch) {
    const int count = batch - at < kF8Batch ? batch - at : kF8Batch;
    Fp8QuantArgs a;
    a.x_dtype = x_dtype;
    a.format = format;
    a.tile = tile;
    a.rows = rows;
    a.cols = cols;
    a.counts = counts;
    a.groups = groups;
    take(a.X, X, at, count);
    take(a.codes, codes, at, count);
    take(a.scales, scales, at, count);
    take(a.codes_t, codes_t, at, count);
    take(a.scales_t, scales_t, at, count);
    if (traced_launch(s, codes_t != nullptr || tile ? "fp8_tile_kernel" : "fp8_rows_kernel", "fp8_quantize", 0.0, bytes * count,
                      [&] { return launch_fp8_quantize(a, count, s); }) != hipSuccess)
      return MUON_ERR_HIP;
  }
  return MUON_OK;
}

muon_status muon_fp8_dequantize(int batch, int rows, int cols, const void* const* codes, const void* const* scales,
                                muon_fp8_format format, void* const* Y, muon_dtype y_dtype, void* stream) {
  if (!shape_ok(batch, rows, cols) || !pointers_ok(batch, codes, kAlign) || !pointers_ok(batch, scales, kAlign) ||
      !pointers_ok(batch, Y))
    return MUON_ERR_INVALID_ARG;
  if (!type_ok(y_dtype) || !format_ok(format) || codes == scales || static_cast<const void*>(codes) == Y ||
      static_cast<const void*>(scales) == Y)
    return MUON_ERR_INVALID_ARG;
  if (y_dtype == MUON_F16) return MUON_ERR_UNSUPPORTED;  // the code's range is that of binary32
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const double bytes = static_cast<double>(rows) * cols * size_of(y_dtype) + code_bytes(rows, fp8_units(cols));
  for (int at = 0; at < batch; at += kF8Batch) {
    const int count = batch - at < kF8Batch ? batch - at : kF8Batch;
    Fp8DequantArgs a;
    a.rows = rows;
    a.cols = cols;
    a.format = format;
    a.y_dtype = y_dtype;
    take(a.codes, codes, at, count);
    take(a.scales, scales, at, count);
    take(a.Y, Y, at, count);
    if (traced_launch(s, "fp8_values_kernel", "fp8_dequantize", 0.0, bytes * count,
                      [&] { return launch_fp8_dequantize(a, count, s); }) != hipSuccess)
      return MUON_ERR_HIP;
  }
  return MUON_OK;
}

size_t muon_fp8_workspace_size(int batch, int m, int n, int k) {
  if (!shape_ok(batch, m, k) || !shape_ok(batch, n, k) || !grid_ok(batch < kF8Batch ? batch : kF8Batch, m, n)) return 0;
  // one launch at a time uses it: the largest need is that of a whole launch or of the last one
  const int whole = batch < kF8Batch ? batch : kF8Batch, rest = batch % kF8Batch;
  size_t bytes = fp8_plan(whole, m, n, k).bytes;
  if (rest > 0) {
    const size_t last = fp8_plan(rest, m, n, k).bytes;
    bytes = last > bytes ? last : bytes;
  }
  return bytes > 256 ? (bytes + 255) / 256 * 256 : 256;
}

muon_status muon_fp8_matmul(int batch, int m, int n, int k, const void* const* A_codes, const void* const* A_scales,
                            muon_fp8_format a_format, const void* const* B_codes, const void* const* B_scales,
                            void* const* C, muon_dtype c_dtype, int accumulate, void* workspace, size_t ws_bytes,
                            void* stream) {
  const size_t need = muon_fp8_workspace_size(batch, m, n, k);
  if (need == 0 || !format_ok(a_format)) return MUON_ERR_INVALID_ARG;
  const void* const* in[4] = {A_codes, A_scales, B_codes, B_scales};
  if (!pointers_ok(batch, C)) return MUON_ERR_INVALID_ARG;
  for (int i = 0; i < 4; ++i)  // A and B may be one matrix (A A^T); C is written
    if (!pointers_ok(batch, in[i], kAlign) || static_cast<const void*>(in[i]) == C) return MUON_ERR_INVALID_ARG;
  if (!type_ok(c_dtype) || (accumulate != 0 && accumulate != 1)) return MUON_ERR_INVALID_ARG;
  if (c_dtype == MUON_F16) return MUON_ERR_UNSUPPORTED;
  if (workspace == nullptr || ws_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return MUON_ERR_WORKSPACE;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const double mn = static_cast<double>(m) * n, units = static_cast<double>(fp8_units(k));
  const double bytes = code_bytes(m, units) + code_bytes(n, units) + mn * size_of(c_dtype) * (accumulate ? 2.0 : 1.0);
  for (int at = 0; at < batch; at += kF8Batch) {
    const int count = batch - at < kF8Batch ? batch - at : kF8Batch;
    const Fp8Plan plan = fp8_plan(count, m, n, k);
    Fp8GemmArgs a;
    a.batch = count;
    a.m = m;
    a.n = n;
    a.units = static_cast<int>(fp8_units(k));
    a.a_format = a_format;
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
    if (traced_launch(s, kernel_name(plan.kind, "fp8_few_rows_kernel", "fp8_tile_gemm_kernel"), "fp8_matmul",
                      2.0 * count * mn * k, bytes * count, [&] { return launch_fp8_gemm(a, plan.kind, s); }) != hipSuccess)
      return MUON_ERR_HIP;
    if (plan.pieces > 1 &&
        traced_launch(s, "fp8_join_kernel", "fp8_join", 0.0, count * mn * (4.0 * plan.pieces + size_of(c_dtype)),
                      [&] { return launch_fp8_join(a, s); }) != hipSuccess)
      return MUON_ERR_HIP;
  }
  return MUON_OK;
}

muon_status muon_fp8_grouped_matmul(int groups, int rows, int n, int k, const int32_t* counts, const void* A_codes,
                                    const void* A_scales, muon_fp8_format a_format, const void* const* B_codes,
                                    const void* const* B_scales, void* C, muon_dtype c_dtype, int accumulate,
                                    int clear_rest, void* stream) {
  if (!shape_ok(1, rows, k) || !shape_ok(1, n, k) || !groups_ok(counts, groups, rows) || !format_ok(a_format) ||
      !grid_ok(1, static_cast<int64_t>(rows) + 64 * (kF8Groups + 1), n))
    return MUON_ERR_INVALID_ARG;
  if (!pointer_ok(A_codes, kAlign) || !pointer_ok(A_scales, kAlign) || !pointers_ok(groups, B_codes, kAlign) ||
      !pointers_ok(groups, B_scales, kAlign) || C == nullptr || C == A_codes || C == A_scales)
    return MUON_ERR_INVALID_ARG;
  if (!type_ok(c_dtype) || (accumulate != 0 && accumulate != 1) || (clear_rest != 0 && clear_rest != 1))
    return MUON_ERR_INVALID_ARG;
  if (c_dtype == MUON_F16) return MUON_ERR_UNSUPPORTED;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const Fp8Kind kind = fp8_row_group_kind(groups, rows, n, k);
  for (int at = 0; at < groups; at += kF8Groups) {
    Fp8RowGroupArgs a;
    a.count = groups - at < kF8Groups ? groups - at : kF8Groups;
    a.m = rows;
    a.n = n;
    a.units = static_cast<int>(fp8_units(k));
    a.a_format = a_format;
    a.c_dtype = c_dtype;
    a.accumulate = accumulate;
    a.clear = clear_rest && at + a.count == groups ? 1 : 0;
    a.groups = groups;
    a.first = at;
    a.counts = counts;
    a.A = A_codes;
    a.As = A_scales;
    a.C = C;
    take(a.B, B_codes, at, a.count);
    take(a.Bs, B_scales, at, a.count);
    // the trace knows no counts: the work is that of all rows, shared by the launches
    const double share = static_cast<double>(a.count) / groups, mn = static_cast<double>(rows) * n;
    const double bytes = (code_bytes(rows, a.units) + mn * size_of(c_dtype) * (accumulate ? 2.0 : 1.0)) * share +
                         code_bytes(n, a.units) * a.count;
    if (traced_launch(s, "fp8_row_groups_kernel", "fp8_grouped_matmul", 2.0 * mn * k * share, bytes,
                      [&] { return launch_fp8_row_groups(a, kind, s); }) != hipSuccess)
      return MUON_ERR_HIP;
  }
  return MUON_OK;
}

muon_status muon_fp8_grouped_weight_grad(int groups, int rows, int m, int n, const int32_t* counts, const void* A_codes,
                                         const void* A_scales, muon_fp8_format a_format, const void* B_codes,
                                         const void* B_scales, void* const* C, muon_dtype c_dtype, int accumulate,
                                         void* stream) {
  if (!shape_ok(1, m, rows) || !shape_ok(1, n, rows) || !groups_ok(counts, groups, rows) || !format_ok(a_format) ||
      !grid_ok(kF8Groups, m, n))
    return MUON_ERR_INVALID_ARG;
  const void* in[4] = {A_codes, A_scales, B_codes, B_scales};
  if (!pointers_ok(groups, C)) return MUON_ERR_INVALID_ARG;
  for (const void* p : in)
    if (!pointer_ok(p, kAlign)) return MUON_ERR_INVALID_ARG;
  if (!type_ok(c_dtype) || (accumulate != 0 && accumulate != 1)) return MUON_ERR_INVALID_ARG;
  if (c_dtype == MUON_F16) return MUON_ERR_UNSUPPORTED;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const Fp8Kind kind = fp8_k_group_kind(groups, rows, m, n, c_dtype == MUON_F32);
  for (int at = 0; at < groups; at += kF8Groups) {
    Fp8KGroupArgs a;
    a.count = groups - at < kF8Groups ? groups - at : kF8Groups;
    a.m = m;
    a.n = n;
    a.rows = rows;
    a.units = static_cast<int>(fp8_group_units(rows, groups));
    a.a_format = a_format;
    a.c_dtype = c_dtype;
    a.accumulate = accumulate;
    a.groups = groups;
    a.first = at;
    a.counts = counts;
    a.A = A_codes;
    a.As = A_scales;
    a.B = B_codes;
    a.Bs = B_scales;
    take(a.C, C, at, a.count);
    const double share = static_cast<double>(a.count) / groups, mn = static_cast<double>(m) * n;
    const double bytes = (code_bytes(m, fp8_units(rows)) + code_bytes(n, fp8_units(rows))) * share +
                         a.count * mn * size_of(c_dtype) * (accumulate ? 2.0 : 1.0);
    if (traced_launch(s, "fp8_k_groups_kernel", "fp8_weight_grad", 2.0 * mn * rows * share, bytes,
                      [&] { return launch_fp8_k_groups(a, kind, s); }) != hipSuccess)
      return MUON_ERR_HIP;
  }
  return MUON_OK;
}

}  // extern "C"

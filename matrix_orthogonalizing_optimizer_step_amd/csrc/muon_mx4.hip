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

constexpr int kThreads = 256;
constexpr int kMaxBlocks = 1 << 16;

// e2m1 code of x times a power of two: y in [0, 8) after scaling.
__device__ __forceinline__ uint32_t e2m1_code(float x, float inverse) {
  const float y = fabsf(x) * inverse;
  const float c = y < 2.0f ? rintf(y * 2.0f) : (y < 4.0f ? rintf(y) + 2.0f : fminf(rintf(y * 0.5f), 3.0f) + 4.0f);
  return static_cast<uint32_t>(c) | ((__float_as_uint(x) >> 28) & 8u);
}

__device__ __forceinline__ float e2m1_value(uint32_t c) {
  const uint32_t e = (c >> 1) & 3u, m = c & 1u;
  const float mag = e == 0u ? 0.5f * static_cast<float>(m)
                            : __uint_as_float(((126u + e) << 23) | (m << 22));
  return (c & 8u) ? -mag : mag;
}

// 2^(127 - byte); byte is at most 252.
__device__ __forceinline__ float scale_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

__device__ __forceinline__ uint32_t max_bits(uint32_t top, float x) {
  const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
  return b > top ? b : top;
}

// Codes along the rows of X: a thread takes 8 elements, 4 threads a block, 16
// a unit; consecutive threads write consecutive bytes.
template <int D>
__global__ __launch_bounds__(kThreads) void mx4_rows_kernel(Mx4QuantArgs a, int64_t units) {
  const void* X = a.X[blockIdx.z];
  uint32_t* codes = static_cast<uint32_t*>(a.codes[blockIdx.z]);
  uint8_t* scales = static_cast<uint8_t*>(a.scales[blockIdx.z]);
  const int64_t total = units * a.rows * 16, step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t id = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; id < total; id += step) {
    const int64_t line = id >> 4;  // u rows + r
    const int64_t u = line / a.rows, r = line - u * a.rows;
    const int64_t c0 = u * kMxUnit + 8 * (id & 15);
    float x[8];
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = c0 + e < a.cols ? load_as_f32(X, r * a.cols + c0 + e, D) : 0.0f;
      top = max_bits(top, x[e]);
    }
    // total is a multiple of 16, so the 4 threads of a block are here together
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      const uint32_t y = static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d));
      top = y > top ? y : top;
    }
    const uint32_t byte = mx4_scale_byte(top);
    uint32_t code = 0;
    if (byte != 255u) {
      const float inv = scale_inverse(byte);
#pragma unroll
      for (int e = 0; e < 8; ++e) code |= e2m1_code(x[e], inv) << (4 * e);
    }
    codes[id] = code;
    if ((id & 3) == 0) scales[id >> 2] = static_cast<uint8_t>(byte);
  }
}

// Codes along the columns of X (the code of X^T): a thread takes one block of
// 32 rows of a column; consecutive threads take consecutive columns.
template <int D>
__global__ __launch_bounds__(kThreads) void mx4_columns_kernel(Mx4QuantArgs a, int64_t units) {
  const void* X = a.X[blockIdx.z];
  uint4* codes = static_cast<uint4*>(a.codes_t[blockIdx.z]);
  uint8_t* scales = static_cast<uint8_t*>(a.scales_t[blockIdx.z]);
  const int64_t total = units * 4 * a.cols, step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t id = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; id < total; id += step) {
    const int64_t block = id / a.cols, j = id - block * a.cols;  // block of 32 rows, column
    const int64_t r0 = block * kMxBlock;
    float x[kMxBlock];
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < kMxBlock; ++e) {
      x[e] = r0 + e < a.rows ? load_as_f32(X, (r0 + e) * a.cols + j, D) : 0.0f;
      top = max_bits(top, x[e]);
    }
    const uint32_t byte = mx4_scale_byte(top);
    uint32_t w[4] = {0, 0, 0, 0};
    if (byte != 255u) {
      const float inv = scale_inverse(byte);
#pragma unroll
      for (int e = 0; e < kMxBlock; ++e) w[e >> 3] |= e2m1_code(x[e], inv) << (4 * (e & 7));
    }
    const int64_t at = ((block >> 2) * a.cols + j) * 4 + (block & 3);
    codes[at] = make_uint4(w[0], w[1], w[2], w[3]);
    scales[at] = static_cast<uint8_t>(byte);
  }
}

// Values of the code, row-major: a thread takes 8 elements of a row.
template <int D>
__global__ __launch_bounds__(kThreads) void mx4_values_kernel(Mx4DequantArgs a, int64_t octets) {
  const uint32_t* codes = static_cast<const uint32_t*>(a.codes[blockIdx.z]);
  const uint8_t* scales = static_cast<const uint8_t*>(a.scales[blockIdx.z]);
  void* Y = a.Y[blockIdx.z];
  const int64_t total = octets * a.rows, step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t id = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; id < total; id += step) {
    const int64_t r = id / octets, o = id - r * octets;
    const int64_t line = (o >> 4) * a.rows + r;
    const uint32_t code = codes[line * 16 + (o & 15)];
    const float s = e8m0_to_f32(scales[line * 4 + ((o & 15) >> 2)]);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (o * 8 + e < a.cols) store_from_f32(Y, r * a.cols + o * 8 + e, D, e2m1_value((code >> (4 * e)) & 15u) * s);
  }
}

uint32_t grid_for(int64_t threads) {
  const int64_t b = (threads + kThreads - 1) / kThreads;
  return static_cast<uint32_t>(b < kMaxBlocks ? b : kMaxBlocks);
}

template <int D>
void quantize(const Mx4QuantArgs& a, int batch, hipStream_t s) {
  if (a.codes[0] != nullptr) {
    const int64_t units = mx4_units(a.cols);
    hipLaunchKernelGGL(mx4_rows_kernel<D>, dim3(grid_for(units * a.rows * 16), 1, batch), dim3(kThreads), 0, s, a, units);
  }
  if (a.codes_t[0] != nullptr) {
    const int64_t units = mx4_units(a.rows);
    hipLaunchKernelGGL(mx4_columns_kernel<D>, dim3(grid_for(units * 4 * a.cols), 1, batch), dim3(kThreads), 0, s, a,
                       units);
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
  const int64_t octets = (static_cast<int64_t>(a.cols) + 7) / 8;
  const dim3 grid(grid_for(octets * a.rows), 1, batch), block(kThreads);
  if (a.y_dtype == kF32) {
    hipLaunchKernelGGL(mx4_values_kernel<kF32>, grid, block, 0, s, a, octets);
  } else {
    hipLaunchKernelGGL(mx4_values_kernel<kBF16>, grid, block, 0, s, a, octets);
  }
  return hipGetLastError();
}

}  // namespace muon

using namespace muon;

namespace {

bool mx4_shape_ok(int batch, int rows, int cols) {
  return batch >= 1 && rows >= 1 && cols >= 1 && rows <= MUON_MAX_DIM && cols <= MUON_MAX_DIM;
}

// A host array of `batch` non-null device pointers.
bool pointers_ok(int batch, const void* const* p) {
  if (p == nullptr) return false;
  for (int i = 0; i < batch; ++i)
    if (p[i] == nullptr) return false;
  return true;
}

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
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < i; ++j)
      if (arrays[i] != nullptr && arrays[i] == arrays[j]) return MUON_ERR_INVALID_ARG;
    if ((i == 0 || arrays[i] != nullptr) && !pointers_ok(batch, arrays[i])) return MUON_ERR_INVALID_ARG;
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
    if (traced_launch(s, "mx4_quantize", "mx4_quantize", 0.0, bytes * count,
                      [&] { return launch_mx4_quantize(a, count, s); }) != hipSuccess)
      return MUON_ERR_HIP;
  }
  return MUON_OK;
}

muon_status muon_mx4_dequantize(int batch, int rows, int cols, const void* const* codes, const void* const* scales,
                                void* const* Y, muon_dtype y_dtype, void* stream) {
  if (!mx4_shape_ok(batch, rows, cols) || !pointers_ok(batch, codes) || !pointers_ok(batch, scales) ||
      !pointers_ok(batch, Y))
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
  return 256;
}

muon_status muon_mx4_matmul(int batch, int m, int n, int k, const void* const* A_codes, const void* const* A_scales,
                            const void* const* B_codes, const void* const* B_scales, void* const* C,
                            muon_dtype c_dtype, int accumulate, void* workspace, size_t ws_bytes, void* stream) {
  const size_t need = muon_mx4_workspace_size(batch, m, n, k);
  if (need == 0) return MUON_ERR_INVALID_ARG;
  const void* const* in[4] = {A_codes, A_scales, B_codes, B_scales};
  if (!pointers_ok(batch, C)) return MUON_ERR_INVALID_ARG;
  for (const void* const* p : in)  // A and B may be one matrix (A A^T); C is written
    if (!pointers_ok(batch, p) || static_cast<const void*>(p) == C) return MUON_ERR_INVALID_ARG;
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
    Mx4GemmArgs a;
    a.m = m;
    a.n = n;
    a.k = k;
    a.units = static_cast<int>(mx4_units(k));
    a.c_dtype = c_dtype;
    a.accumulate = accumulate;
    take(a.A, A_codes, at, count);
    take(a.As, A_scales, at, count);
    take(a.B, B_codes, at, count);
    take(a.Bs, B_scales, at, count);
    take(a.C, C, at, count);
    if (traced_launch(s, "mx4_gemm_kernel", "mx4_matmul", 2.0 * count * mn * k, bytes * count,
                      [&] { return launch_mx4_gemm(a, count, s); }) != hipSuccess)
      return MUON_ERR_HIP;
  }
  return MUON_OK;
}

}  // extern "C"

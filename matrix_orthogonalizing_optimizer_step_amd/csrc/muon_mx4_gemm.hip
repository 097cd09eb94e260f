// C = A B^T (+ C) of two matrices in the microscaled 4-bit code, on the
// block-scaled MFMA (v_mfma_scale_f32_32x32x64_f8f6f4 with fp4 operands): a
// lane holds one block of 32 elements of one row, 16 bytes, and that block's
// scale byte; the products and their sum over k are fp32.
//
// The order of k is free as long as A and B agree, so lanes 0..31 take unit
// 2 j and lanes 32..63 unit 2 j + 1 of the row, and the four MFMAs of a pair of
// units take blocks 0..3 of each: a lane reads 64 consecutive code bytes and
// one 32-bit word of scales for them.
#include "muon_convert.h"
#include "muon_internal.h"
#include "muon_mx4.h"

namespace muon {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr int kFp4 = 4;  // the operand format field of the MFMA

template <int S>
__device__ __forceinline__ f32x16_t mfma_mx4(const uint4& a, const uint4& b, const f32x16_t& c, uint32_t sa, uint32_t sb) {
  const i32x8_t av = {static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z), static_cast<int>(a.w), 0, 0, 0, 0};
  const i32x8_t bv = {static_cast<int>(b.x), static_cast<int>(b.y), static_cast<int>(b.z), static_cast<int>(b.w), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, kFp4, kFp4, S, static_cast<int>(sa), S,
                                                         static_cast<int>(sb));
}

constexpr int kTile = 64;  // block tile edge: 4 waves, one 32 x 32 MFMA tile each

template <int DC>
__global__ __launch_bounds__(256) void mx4_gemm_kernel(Mx4GemmArgs a) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int i0 = blockIdx.y * kTile + 32 * (wave >> 1), j0 = blockIdx.x * kTile + 32 * (wave & 1);
  const int b = blockIdx.z;
  const uint4* A = static_cast<const uint4*>(a.A[b]);
  const uint4* B = static_cast<const uint4*>(a.B[b]);
  const uint32_t* As = static_cast<const uint32_t*>(a.As[b]);
  const uint32_t* Bs = static_cast<const uint32_t*>(a.Bs[b]);
  const int ra = i0 + (lane & 31), rb = j0 + (lane & 31);
  f32x16_t acc = {};
  for (int u0 = 0; u0 < a.units; u0 += 2) {
    const int u = u0 + (lane >> 5);
    uint4 av[4] = {}, bv[4] = {};
    uint32_t sa = 0, sb = 0;
    if (u < a.units && ra < a.m) {
      const int64_t line = static_cast<int64_t>(u) * a.m + ra;
      for (int s = 0; s < 4; ++s) av[s] = A[line * 4 + s];
      sa = As[line];
    }
    if (u < a.units && rb < a.n) {
      const int64_t line = static_cast<int64_t>(u) * a.n + rb;
      for (int s = 0; s < 4; ++s) bv[s] = B[line * 4 + s];
      sb = Bs[line];
    }
    acc = mfma_mx4<0>(av[0], bv[0], acc, sa, sb);
    acc = mfma_mx4<1>(av[1], bv[1], acc, sa, sb);
    acc = mfma_mx4<2>(av[2], bv[2], acc, sa, sb);
    acc = mfma_mx4<3>(av[3], bv[3], acc, sa, sb);
  }
  void* C = a.C[b];
  const int j = j0 + (lane & 31);
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int i = i0 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
    if (i < a.m && j < a.n) {
      const int64_t at = static_cast<int64_t>(i) * a.n + j;
      const float c = a.accumulate ? load_as_f32(C, at, DC) + acc[r] : acc[r];
      store_from_f32(C, at, DC, c);
    }
  }
}

}  // namespace

hipError_t launch_mx4_gemm(const Mx4GemmArgs& a, int batch, hipStream_t s) {
  const dim3 grid((a.n + kTile - 1) / kTile, (a.m + kTile - 1) / kTile, batch), block(256);
  if (a.c_dtype == kF32) {
    hipLaunchKernelGGL(mx4_gemm_kernel<kF32>, grid, block, 0, s, a);
  } else {
    hipLaunchKernelGGL(mx4_gemm_kernel<kBF16>, grid, block, 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace muon

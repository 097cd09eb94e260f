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

// ---------------------------------------------------------------------------
// 256 x 256 tiles: 4 waves of 128 x 128 (4 x 4 MFMA tiles, 256 accumulators),
// one block per compute unit.  k runs in slabs of one unit (128): the tile's
// codes (2 x 16 KB, each one contiguous piece of memory) and scales (2 x 1 KB)
// go straight into a ring of 4 LDS stages, three slabs ahead.  Lanes 0..31
// take blocks 0 and 1 of the unit, lanes 32..63 blocks 2 and 3 (two MFMAs per
// tile and slab).  Block b of row r lies in slot b ^ (r / 4 % 4) of the row's 64
// bytes, so that 16 lanes reading one block of 16 rows touch all LDS banks
// once; the permutation is in the global addresses of the loads, which stay
// within a row's 64 bytes.
//
// The fragments of a k-step are read while the previous step's MFMAs run.  The
// barrier sits in the middle of a slab's second step: all reads of the slab are
// done by then, so its stage can be filled anew, and the step's other half
// covers the first reads of the next slab.
// ---------------------------------------------------------------------------
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int kBig = 256;                          // tile edge
constexpr int kStages = 4;
constexpr int kStageU4 = 2 * kBig * 4;             // uint4 of codes per stage
constexpr int kSchedMfma = 0x008, kSchedVmem = 0x010, kSchedDsRead = 0x100;  // sched_group_barrier masks
constexpr int kLoadsPerSlab = 10;                  // per wave: 4 + 4 of codes, 1 + 1 of scales

struct BigStage {
  uint4 code[kStageU4];        // A rows, then B rows, 4 slots each
  uint32_t scale[2 * kBig];    // A rows, then B rows
};

constexpr int waitcnt_imm(int vm, int lgkm) {  // vmcnt, no wait for exports, lgkmcnt
  return (vm & 15) | (((vm >> 4) & 3) << 14) | (7 << 4) | ((lgkm & 15) << 8);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  const uint64_t u = reinterpret_cast<uint64_t>(base);
  const uint64_t lo = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(u & 0xffffffffu)));
  const uint64_t hi = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(u >> 32)));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(lo | (hi << 32)), static_cast<short>(0),
                                           __builtin_amdgcn_readfirstlane(static_cast<int>(bytes)), 0x00020000);
}

// One operand's source: codes and scales of the 64 rows this wave loads.
struct BigSource {
  __amdgpu_buffer_rsrc_t code, scale;
  uint32_t row;     // first row of this wave's loads
  uint32_t rows;    // rows of the matrix
};

__device__ __forceinline__ void load_operand(BigStage& st, int side, const BigSource& src, uint32_t u, int wave,
                                             int vcode, int vscale) {
  // u may lie behind the last unit and rows behind the last row: such addresses
  // are behind the buffer's end (zeros) or in the next unit's rows, and what
  // they give enters no stored element
  const uint32_t line = u * src.rows + src.row;
  const int so = __builtin_amdgcn_readfirstlane(static_cast<int>(line * 64u));
  lds_ptr_t dst = (lds_ptr_t)(st.code + (side * kBig + wave * 64) * 4);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(src.code, dst, 16, vcode, so, 0, 0);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(src.code, dst, 16, vcode, so, 1024, 0);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(src.code, dst, 16, vcode, so, 2048, 0);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(src.code, dst, 16, vcode, so, 3072, 0);
  lds_ptr_t sd = (lds_ptr_t)(st.scale + side * kBig + wave * 64);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(src.scale, sd, 4, vscale,
                                           __builtin_amdgcn_readfirstlane(static_cast<int>(line * 4u)), 0, 0);
}

struct Frags {
  uint4 a[4], b[4];
};
struct ScaleWords {
  uint32_t a[4], b[4];
};

// k-step s of a stage: this wave's 4 row fragments of A and of B.
__device__ __forceinline__ void read_frag(uint4 (&f)[4], const BigStage& st, int first_row, int lane, int s) {
  const int r = lane & 31, slot = (2 * (lane >> 5) + s) ^ ((r >> 2) & 3);
#pragma unroll
  for (int x = 0; x < 4; ++x) f[x] = st.code[(first_row + 32 * x + r) * 4 + slot];
}
__device__ __forceinline__ void read_scales(uint32_t (&w)[4], const BigStage& st, int first_row, int lane) {
#pragma unroll
  for (int x = 0; x < 4; ++x) w[x] = st.scale[first_row + 32 * x + (lane & 31)];
}
// The upper lanes' blocks are bytes 2 and 3.
__device__ __forceinline__ void shift_scales(uint32_t (&w)[4], int lane) {
#pragma unroll
  for (int x = 0; x < 4; ++x) w[x] >>= (lane >> 5) * 16;
}

template <int S, int Y0, int Y1>
__device__ __forceinline__ void mfmas(f32x16_t (&acc)[4][4], const Frags& f, const ScaleWords& w) {
#pragma unroll
  for (int y = Y0; y < Y1; ++y)
#pragma unroll
    for (int x = 0; x < 4; ++x) acc[x][y] = mfma_mx4<S>(f.b[x], f.a[y], acc[x][y], w.b[x], w.a[y]);
}

// One slab from stage `cur`; fragments of its first step are in f0, its scales
// in w.  Ends with those of the next slab (stage `nxt`) there.
__device__ __forceinline__ void slab(f32x16_t (&acc)[4][4], Frags& f0, ScaleWords& w, BigStage& cur,
                                     const BigStage& nxt, const BigSource& A, const BigSource& B, uint32_t u, int wave,
                                     int lane, int vcode, int vscale, int ra, int rb) {
  Frags f1;
  read_frag(f1.b, cur, rb, lane, 1);
  read_frag(f1.a, cur, ra, lane, 1);
  mfmas<0, 0, 4>(acc, f0, w);
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    __builtin_amdgcn_sched_group_barrier(kSchedDsRead, 1, 0);
    __builtin_amdgcn_sched_group_barrier(kSchedMfma, 2, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
  mfmas<1, 0, 2>(acc, f1, w);
  // this wave's part of the next slab has landed (two slabs stay in flight), and
  // all its reads of this one are done
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(2 * kLoadsPerSlab, 0));
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  load_operand(cur, 0, A, u + kStages, wave, vcode, vscale);
  load_operand(cur, 1, B, u + kStages, wave, vcode, vscale);
  ScaleWords wn;
  read_frag(f0.b, nxt, rb, lane, 0);
  read_frag(f0.a, nxt, ra, lane, 0);
  read_scales(wn.b, nxt, rb, lane);
  read_scales(wn.a, nxt, ra, lane);
  mfmas<1, 2, 4>(acc, f1, w);
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
    __builtin_amdgcn_sched_group_barrier(kSchedDsRead, 2, 0);
    __builtin_amdgcn_sched_group_barrier(kSchedVmem, 2, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
  shift_scales(wn.b, lane);
  shift_scales(wn.a, lane);
  w = wn;
}

// Block id -> tile: consecutive ids go to the 8 XCDs in turn, so each XCD gets a
// contiguous range of tiles, and tiles run down columns of 4 tile rows, so that
// the tiles an XCD works on at one time share their rows of A and B in its L2.
__device__ __forceinline__ void tile_of(int id, int total, int tm, int tn, int* batch, int* ti, int* tj) {
  const int q = total >> 3, rest = total & 7, x = id & 7, at = id >> 3;
  int t = x * q + (x < rest ? x : rest) + at;
  const int per = tm * tn;
  *batch = t / per;
  t -= *batch * per;
  constexpr int kGroup = 4;
  const int g = t / (kGroup * tn), first = g * kGroup, h = tm - first < kGroup ? tm - first : kGroup;
  t -= g * kGroup * tn;
  *ti = first + t % h;
  *tj = t / h;
}

template <int DC>
__device__ __forceinline__ void store_quad(void* C, int64_t at, const float (&v)[4], int left, bool vec, int accumulate) {
  float x[4] = {v[0], v[1], v[2], v[3]};
  if (vec && left >= 4) {
    if constexpr (DC == kF32) {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(C) + at);
      if (accumulate) {
        const float4 c = *p;
        x[0] += c.x; x[1] += c.y; x[2] += c.z; x[3] += c.w;
      }
      *p = make_float4(x[0], x[1], x[2], x[3]);
    } else {
      uint2* p = reinterpret_cast<uint2*>(static_cast<uint16_t*>(C) + at);
      if (accumulate) {
        const uint2 c = *p;
        x[0] += bf16_to_f32(static_cast<uint16_t>(c.x));
        x[1] += bf16_to_f32(static_cast<uint16_t>(c.x >> 16));
        x[2] += bf16_to_f32(static_cast<uint16_t>(c.y));
        x[3] += bf16_to_f32(static_cast<uint16_t>(c.y >> 16));
      }
      *p = make_uint2(f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) store_from_f32(C, at + e, DC, accumulate ? load_as_f32(C, at + e, DC) + x[e] : x[e]);
  }
}

template <int DC>
__global__ __launch_bounds__(256, 1) void mx4_gemm_big_kernel(Mx4GemmArgs a, int tm, int tn) {
  __shared__ BigStage s0, s1, s2, s3;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)), lane = threadIdx.x & 63;
  int b, ti, tj;
  tile_of(blockIdx.x, gridDim.x, tm, tn, &b, &ti, &tj);
  const int i0 = ti * kBig, j0 = tj * kBig;
  const uint32_t lines_a = static_cast<uint32_t>(a.units) * a.m, lines_b = static_cast<uint32_t>(a.units) * a.n;
  const BigSource A{make_rsrc(a.A[b], lines_a * 64u), make_rsrc(a.As[b], lines_a * 4u),
                    static_cast<uint32_t>(i0 + wave * 64), static_cast<uint32_t>(a.m)};
  const BigSource B{make_rsrc(a.B[b], lines_b * 64u), make_rsrc(a.Bs[b], lines_b * 4u),
                    static_cast<uint32_t>(j0 + wave * 64), static_cast<uint32_t>(a.n)};
  // lane l fills slot l % 4 of row l / 4 of each 16-row piece
  const int vcode = (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 4) & 3)) * 16), vscale = lane * 4;
  BigStage* st[kStages] = {&s0, &s1, &s2, &s3};
#pragma unroll
  for (int s = 0; s < kStages; ++s) {
    load_operand(*st[s], 0, A, s, wave, vcode, vscale);
    load_operand(*st[s], 1, B, s, wave, vcode, vscale);
  }
  const int ra = 128 * (wave >> 1), rb = kBig + 128 * (wave & 1);
  f32x16_t acc[4][4] = {};
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(3 * kLoadsPerSlab, 0));
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  Frags f;
  ScaleWords w;
  read_frag(f.b, s0, rb, lane, 0);
  read_frag(f.a, s0, ra, lane, 0);
  read_scales(w.b, s0, rb, lane);
  read_scales(w.a, s0, ra, lane);
  shift_scales(w.b, lane);
  shift_scales(w.a, lane);
  int u = 0;
  for (; u + kStages <= a.units; u += kStages) {
    slab(acc, f, w, s0, s1, A, B, u, wave, lane, vcode, vscale, ra, rb);
    slab(acc, f, w, s1, s2, A, B, u + 1, wave, lane, vcode, vscale, ra, rb);
    slab(acc, f, w, s2, s3, A, B, u + 2, wave, lane, vcode, vscale, ra, rb);
    slab(acc, f, w, s3, s0, A, B, u + 3, wave, lane, vcode, vscale, ra, rb);
  }
  if (u < a.units) slab(acc, f, w, s0, s1, A, B, u, wave, lane, vcode, vscale, ra, rb);
  if (u + 1 < a.units) slab(acc, f, w, s1, s2, A, B, u + 1, wave, lane, vcode, vscale, ra, rb);
  if (u + 2 < a.units) slab(acc, f, w, s2, s3, A, B, u + 2, wave, lane, vcode, vscale, ra, rb);
  // loads behind the last unit are still on their way into LDS: they end before
  // the block does
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
  // D = (B rows) x (A rows): lane l holds row l % 32 of C and, in registers
  // 4 g .. 4 g + 3, columns 8 g + 4 (l / 32) .. + 3
  void* C = a.C[b];
  const bool vec = (a.n & 3) == 0 && (reinterpret_cast<uintptr_t>(C) & (DC == kF32 ? 15u : 7u)) == 0;
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    const int i = i0 + ra + 32 * y + (lane & 31);
    if (i < a.m) {
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int j = j0 + (rb - kBig) + 32 * x + 8 * g + 4 * (lane >> 5);
          const float v[4] = {acc[x][y][4 * g], acc[x][y][4 * g + 1], acc[x][y][4 * g + 2], acc[x][y][4 * g + 3]};
          store_quad<DC>(C, static_cast<int64_t>(i) * a.n + j, v, a.n - j, vec, a.accumulate);
        }
    }
  }
}

}  // namespace

hipError_t launch_mx4_gemm(const Mx4GemmArgs& a, int batch, hipStream_t s) {
  if (a.m > 128 && a.n > 128) {
    const int tm = (a.m + kBig - 1) / kBig, tn = (a.n + kBig - 1) / kBig;
    const dim3 grid(static_cast<uint32_t>(tm) * tn * batch), block(256);
    if (a.c_dtype == kF32) {
      hipLaunchKernelGGL(mx4_gemm_big_kernel<kF32>, grid, block, 0, s, a, tm, tn);
    } else {
      hipLaunchKernelGGL(mx4_gemm_big_kernel<kBF16>, grid, block, 0, s, a, tm, tn);
    }
    return hipGetLastError();
  }
  const dim3 grid((a.n + kTile - 1) / kTile, (a.m + kTile - 1) / kTile, batch), block(256);
  if (a.c_dtype == kF32) {
    hipLaunchKernelGGL(mx4_gemm_kernel<kF32>, grid, block, 0, s, a);
  } else {
    hipLaunchKernelGGL(mx4_gemm_kernel<kBF16>, grid, block, 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace muon

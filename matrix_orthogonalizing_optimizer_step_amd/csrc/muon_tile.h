// Building blocks of the products of coded matrices in MFMA tiles: buffer
// resources, waits, the order of the tiles, and the way of the accumulators to C.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "muon_convert.h"
#include "muon_internal.h"

namespace muon {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int kCUs = 256;  // compute units of the MI355X: plans depend on shapes only
constexpr int kSchedValu = 0x002, kSchedMfma = 0x008, kSchedVmem = 0x010, kSchedDsRead = 0x100;  // sched_group_barrier masks

inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

constexpr int waitcnt_imm(int vm, int lgkm) {  // vmcnt, no wait for exports, lgkmcnt
  return (vm & 15) | (((vm >> 4) & 3) << 14) | (7 << 4) | ((lgkm & 15) << 8);
}

// A buffer resource of `bytes` bytes at `base` + `offset` (all block-uniform).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint64_t offset, uint32_t bytes) {
  const uint64_t u = reinterpret_cast<uint64_t>(base) + offset;
  const uint64_t lo = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(u & 0xffffffffu)));
  const uint64_t hi = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(u >> 32)));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(lo | (hi << 32)), static_cast<short>(0),
                                           __builtin_amdgcn_readfirstlane(static_cast<int>(bytes)), 0x00020000);
}

// Tile t of tm x tn, running down columns of 4 tile rows, so that tiles worked on at
// one time share their rows of A and B in an L2.
__device__ __forceinline__ void tile_in_bands(int t, int tm, int tn, int* ti, int* tj) {
  constexpr int kGroup = 4;
  const int g = t / (kGroup * tn), first = g * kGroup, h = tm - first < kGroup ? tm - first : kGroup;
  t -= g * kGroup * tn;
  *ti = first + t % h;
  *tj = t / h;
}

// Block id -> tile: consecutive ids go to the 8 XCDs in turn, so each XCD gets a
// contiguous range of tiles.
__device__ __forceinline__ void tile_of(int id, int total, int tm, int tn, int* outer, int* ti, int* tj) {
  const int q = total >> 3, rest = total & 7, x = id & 7, at = id >> 3;
  int t = x * q + (x < rest ? x : rest) + at;
  const int per = tm * tn;
  *outer = t / per;
  t -= *outer * per;
  tile_in_bands(t, tm, tn, ti, tj);
}

// Four consecutive elements of a row of C (those with left > 0), with what is
// there if asked for.  vec: the place is aligned to four elements.
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

typedef u32x4_t u32x4_a2 __attribute__((aligned(2)));

// A wave's accumulators to C, 32 rows at a time through its own LDS (`stage`).
// With D = (B rows) x (A rows) lane l holds row l % 32 of C and, in registers 4 g
// .. 4 g + 3, columns 8 g + 4 (l / 32) .. + 3 of an MFMA tile; read back, a lane
// has 16 bytes of a row, so that a store fills whole 128 FN-byte (bf16: 64 FN)
// pieces of rows.  LDS holds C's type, or fp32 where C is added to: C is rounded
// once.  Measured on 8192x7168x3584 against 8-byte stores of 32 rows at a time
// straight from the accumulators: 138 -> 122 us.  XS: columns of MFMA tiles that are
// staged together (the LDS takes 32 rows of them).  FULL: all of the wave's rows and
// columns are there.
//
// Where C is added to, full tiles have what is there on its way kAhead steps ahead of
// its use: loads and stores end in order, so a load behind the stores of the rows before
// would wait for those.  (us, us without: 8-bit products' fp32 G of 16 experts of
// 2048x7168, 8190 rows, 436 / 730, 8192x8192x2048 278 / 358; 4-bit 3584x7168x8192 114 /
// 140.)  Not for bf16 in 256 x 256 tiles: there it takes registers that the products need
// (16 experts 319 / 436, but 274 / 241 where C is not added to).
template <class T, int DC, bool ADD, int XS = T::FN, bool FULL = false>
__device__ __forceinline__ void store_tile(void* C, const f32x16_t (&acc)[T::FN][T::FM], uint4* stage, int i, int j,
                                           int m, int n, int lane) {
  constexpr int kSize = DC == kF32 ? 4 : 2, kHeld = ADD || DC == kF32 ? 4 : 2;  // bytes of an element of C, in LDS
  constexpr int kCols = 32 * XS, kPitch = kCols * kHeld / 16 + 1;            // uint4 of a row, one against conflicts
  constexpr int kLanes = kCols * kSize / 16, kRows = 64 / kLanes;               // lanes of a row, rows of a store
  static_assert(T::FN % XS == 0 && 32 * kPitch * 16 <= sizeof(typename T::Stage) && kLanes <= 64, "staging");
  const int row = lane & 31, half = lane >> 5, r0 = lane / kLanes, chunk = lane % kLanes;
  constexpr int kElems = 16 / kSize;
  if constexpr (ADD && !FULL && (DC == kF32 || T::FM * T::FN < 16)) {
    if (i + 32 * T::FM <= m && j + 32 * T::FN <= n) {
      store_tile<T, DC, ADD, XS, true>(C, acc, stage, i, j, m, n, lane);
      return;
    }
  }
  constexpr int kSteps = T::FM * (T::FN / XS), kLoads = 32 / kRows, kAhead = kLoads < 12 ? 12 / kLoads : 1;
  u32x4_t was[ADD && FULL ? kSteps : 1][kLoads];
  const auto load = [&](int yx) {
    const int y = yx / (T::FN / XS), x0 = yx % (T::FN / XS) * XS;
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const int64_t at = static_cast<int64_t>(i + 32 * y + q * kRows + r0) * n + j + 32 * x0 + chunk * kElems;
      was[yx][q] = *reinterpret_cast<const u32x4_a2*>(static_cast<const char*>(C) + at * kSize);
    }
  };
  if constexpr (ADD && FULL) {
#pragma unroll
    for (int yx = 0; yx < kAhead && yx < kSteps; ++yx) load(yx);
  }
#pragma unroll
  for (int yx = 0; yx < T::FM * (T::FN / XS); ++yx) {
    const int y = yx / (T::FN / XS), x0 = yx % (T::FN / XS) * XS;
    const int jc = j + 32 * x0 + chunk * kElems;
    if constexpr (ADD && FULL)
      if (yx + kAhead < kSteps) load(yx + kAhead);
#pragma unroll
    for (int x = 0; x < XS; ++x)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x16_t& t = acc[x0 + x][y];
        const float v[4] = {t[4 * g], t[4 * g + 1], t[4 * g + 2], t[4 * g + 3]};
        const int col = 32 * x + 8 * g + 4 * half;
        if constexpr (kHeld == 4) {
          stage[row * kPitch + col / 4] = __builtin_bit_cast(uint4, make_float4(v[0], v[1], v[2], v[3]));
        } else {
          reinterpret_cast<uint2*>(stage)[row * kPitch * 2 + col / 4] =
              make_uint2(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]));
        }
      }
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
    asm volatile("" ::: "memory");  // the wave's own writes, in order with its reads
#pragma unroll
    for (int q = 0; q < 32 / kRows; ++q) {
      const int r = q * kRows + r0, ir = i + 32 * y + r;
      if (FULL || (ir < m && jc < n)) {
        char* const p = static_cast<char*>(C) + (static_cast<int64_t>(ir) * n + jc) * kSize;
        float f[kElems];
        uint4 h;
        if constexpr (kHeld == 4) {
#pragma unroll
          for (int e = 0; e < kElems; e += 4) {
            const float4 t = __builtin_bit_cast(float4, stage[r * kPitch + (chunk * kElems + e) / 4]);
            f[e] = t.x; f[e + 1] = t.y; f[e + 2] = t.z; f[e + 3] = t.w;
          }
        } else {
          h = stage[r * kPitch + chunk];
        }
        if (FULL || jc + kElems <= n) {
          if constexpr (kHeld == 4) {
            if constexpr (ADD) {
              u32x4_t c;
              if constexpr (FULL) {
                c = was[yx][q];
              } else {
                c = *reinterpret_cast<const u32x4_a2*>(p);
              }
#pragma unroll
              for (int e = 0; e < kElems; ++e)
                f[e] += DC == kF32 ? __uint_as_float(c[e & 3])
                                   : bf16_to_f32(static_cast<uint16_t>((e & 1) ? c[e >> 1] >> 16 : c[e >> 1]));
            }
            if constexpr (DC == kF32) {
              *reinterpret_cast<u32x4_a2*>(p) = (u32x4_t){__float_as_uint(f[0]), __float_as_uint(f[1]),
                                                          __float_as_uint(f[2]), __float_as_uint(f[3])};
            } else {
              *reinterpret_cast<u32x4_a2*>(p) = (u32x4_t){f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]),
                                                          f32x2_to_bf16x2(f[4], f[5]), f32x2_to_bf16x2(f[6], f[7])};
            }
          } else {
            *reinterpret_cast<u32x4_a2*>(p) = (u32x4_t){h.x, h.y, h.z, h.w};
          }
        } else {
#pragma unroll
          for (int e = 0; e < kElems; ++e)
            if (jc + e < n) {
              if constexpr (kHeld == 4) {
                store_from_f32(p, e, DC, ADD ? load_as_f32(p, e, DC) + f[e] : f[e]);
              } else {
                const uint32_t w = (&h.x)[e >> 1];
                reinterpret_cast<uint16_t*>(p)[e] = static_cast<uint16_t>((e & 1) ? w >> 16 : w);
              }
            }
        }
      }
    }
    asm volatile("" ::: "memory");  // the next rows' writes stay behind these reads
  }
}

}  // namespace muon

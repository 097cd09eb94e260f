// C = A B^T (+ C) of two matrices in the microscaled 4-bit code, on the
// block-scaled MFMA with fp4 operands: a lane holds one block of 32 elements of
// one row, 16 bytes, and that block's scale byte; the products and their sum over
// k are fp32.
//
// The order of k is free as long as A and B agree.  The tiles take 32x32x64 MFMAs,
// two for a unit of 128 (lanes 0..31 blocks 0 and 1 of their row, lanes 32..63
// blocks 2 and 3), through LDS; for at most 16 rows of A a 16x16x128 MFMA takes a
// whole unit (16 lanes a block), straight from memory.
#include "muon_convert.h"
#include "muon_internal.h"
#include "muon_mx4.h"

namespace muon {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kFp4 = 4;  // the operand format field of the MFMA

template <int S>
__device__ __forceinline__ f32x16_t mfma_mx4(const uint4& a, const uint4& b, const f32x16_t& c, uint32_t sa, uint32_t sb) {
  const i32x8_t av = {static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z), static_cast<int>(a.w), 0, 0, 0, 0};
  const i32x8_t bv = {static_cast<int>(b.x), static_cast<int>(b.y), static_cast<int>(b.z), static_cast<int>(b.w), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, kFp4, kFp4, S, static_cast<int>(sa), S,
                                                         static_cast<int>(sb));
}

typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kCUs = 256;  // compute units of the MI355X: the plans below depend on shapes only

// ---------------------------------------------------------------------------
// TM x TN tiles by 4 waves (WM x 4 / WM, each FM x FN MFMA tiles of 32 x 32).  k
// runs in slabs of one unit (128): the tile's codes (each operand one
// contiguous piece of memory) and scales go straight into a ring of 4 LDS
// stages, three slabs ahead.  Lanes 0..31 take blocks 0 and 1 of the unit, lanes
// 32..63 blocks 2 and 3 (two MFMAs per MFMA tile and slab).  Block b of row r
// lies in slot b ^ (r / 4 % 4) of the row's 64 bytes, so that 16 lanes reading
// one block of 16 rows touch all LDS banks once; the permutation is in the
// global addresses of the loads, which stay within a row's 64 bytes.
//
// The fragments of a k-step are read while the previous step's MFMAs run.  The
// barrier sits in the middle of a slab's second step: all reads of the slab are
// done by then, so its stage can be filled anew, and the step's other half
// covers the first reads of the next slab.
// ---------------------------------------------------------------------------
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int kStages = 4;
constexpr int kSchedMfma = 0x008, kSchedVmem = 0x010, kSchedDsRead = 0x100;  // sched_group_barrier masks

template <int TM_, int TN_, int WM_>
struct Tile {
  static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = 4 / WM_;
  static constexpr int FM = TM / WM / 32, FN = TN / WN / 32;
  static constexpr int kLoads = TM / 64 + TN / 64 + 2;  // per wave and slab: codes, and scales of A and B
  static constexpr int kAfter = kLoads / 3;             // of them, right behind the barrier
  struct Stage {
    uint4 code[(TM + TN) * 4];   // A rows, then B rows, 4 slots each
    uint32_t scale[TM + TN];
  };
};

constexpr int waitcnt_imm(int vm, int lgkm) {  // vmcnt, no wait for exports, lgkmcnt
  return (vm & 15) | (((vm >> 4) & 3) << 14) | (7 << 4) | ((lgkm & 15) << 8);
}

// A buffer resource of `bytes` bytes at `base` + `offset` (all block-uniform).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t offset, uint32_t bytes) {
  const uint64_t u = reinterpret_cast<uint64_t>(base) + offset;
  const uint64_t lo = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(u & 0xffffffffu)));
  const uint64_t hi = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(u >> 32)));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(lo | (hi << 32)), static_cast<short>(0),
                                           __builtin_amdgcn_readfirstlane(static_cast<int>(bytes)), 0x00020000);
}

// One operand's source, seen from this lane.
struct Source {
  const void* code;
  const void* scale;
  int vcode, vscale;     // byte offsets of this lane's first loads from a unit's first row
  uint32_t rows, lines;  // rows of the matrix; units x rows
};

// Loads FIRST .. LAST - 1 of the T::kLoads that bring this wave's share of unit u
// into a stage: the codes of A and of B, 16 rows each, and the scales of A and
// of B.  Behind the last unit the last one is read again.  The resource starts at
// the unit and ends with the matrix, so every load is checked against the
// matrix's end: rows behind the last row read the next unit's, or zeros behind
// the last unit.  Neither enters a stored element.
template <class T, int FIRST, int LAST>
__device__ __forceinline__ void load_unit(typename T::Stage& st, const Source& A, const Source& B, int u, int last,
                                          int wave, int lane) {
  constexpr int RA = T::TM / 4, RB = T::TN / 4;  // rows of this wave
  const uint32_t unit = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(u < last ? u : last));
  const uint32_t la = unit * A.rows, lb = unit * B.rows;
  const __amdgpu_buffer_rsrc_t ca = make_rsrc(A.code, la * 64u, (A.lines - la) * 64u);
  const __amdgpu_buffer_rsrc_t cb = make_rsrc(B.code, lb * 64u, (B.lines - lb) * 64u);
  lds_ptr_t da = (lds_ptr_t)(st.code + wave * RA * 4), db = (lds_ptr_t)(st.code + (T::TM + wave * RB) * 4);
#define MX4_LOAD(N, R, RSRC, DST, VOFF, PIECE)                            \
  if constexpr (FIRST <= (N) && (N) < LAST && (PIECE) * 1024 < (R) * 64)  \
    __builtin_amdgcn_raw_ptr_buffer_load_lds(RSRC, DST, 16, VOFF, 0, (PIECE) * 1024, 0)
  constexpr int NA = RA / 16, NB = RB / 16;
  MX4_LOAD(0, RA, ca, da, A.vcode, 0);
  MX4_LOAD(1, RA, ca, da, A.vcode, 1);
  MX4_LOAD(2, RA, ca, da, A.vcode, 2);
  MX4_LOAD(3, RA, ca, da, A.vcode, 3);
  MX4_LOAD(NA, RB, cb, db, B.vcode, 0);
  MX4_LOAD(NA + 1, RB, cb, db, B.vcode, 1);
  MX4_LOAD(NA + 2, RB, cb, db, B.vcode, 2);
  MX4_LOAD(NA + 3, RB, cb, db, B.vcode, 3);
#undef MX4_LOAD
  static_assert(RA <= 64 && RB <= 64 && NA + NB + 2 == T::kLoads, "loads of a unit");
  if constexpr (FIRST <= NA + NB && NA + NB < LAST) {
    if (RA == 64 || lane < RA)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(A.scale, la * 4u, (A.lines - la) * 4u),
                                               (lds_ptr_t)(st.scale + wave * RA), 4, A.vscale, 0, 0, 0);
  }
  if constexpr (FIRST <= NA + NB + 1 && NA + NB + 1 < LAST) {
    if (RB == 64 || lane < RB)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(B.scale, lb * 4u, (B.lines - lb) * 4u),
                                               (lds_ptr_t)(st.scale + T::TM + wave * RB), 4, B.vscale, 0, 0, 0);
  }
}

// The 32-row fragments of k-step s from row `first` of a stage on.
template <int F, class Stage>
__device__ __forceinline__ void read_frag(uint4 (&f)[F], const Stage& st, int first, int lane, int s) {
  const int r = lane & 31, slot = (2 * (lane >> 5) + s) ^ ((r >> 2) & 3);
#pragma unroll
  for (int x = 0; x < F; ++x) f[x] = st.code[(first + 32 * x + r) * 4 + slot];
}
template <int F, class Stage>
__device__ __forceinline__ void read_scales(uint32_t (&w)[F], const Stage& st, int first, int lane) {
#pragma unroll
  for (int x = 0; x < F; ++x) w[x] = st.scale[first + 32 * x + (lane & 31)];
}
// The upper lanes' blocks are bytes 2 and 3.
template <int F>
__device__ __forceinline__ void shift_scales(uint32_t (&w)[F], int lane) {
#pragma unroll
  for (int x = 0; x < F; ++x) w[x] >>= (lane >> 5) * 16;
}

template <class T>
struct Frags {
  uint4 a[T::FM], b[T::FN];
};
template <class T>
struct ScaleWords {
  uint32_t a[T::FM], b[T::FN];
};

template <class T, int S, int Y0, int Y1>
__device__ __forceinline__ void mfmas(f32x16_t (&acc)[T::FN][T::FM], const Frags<T>& f, const ScaleWords<T>& w) {
#pragma unroll
  for (int y = Y0; y < Y1; ++y)
#pragma unroll
    for (int x = 0; x < T::FN; ++x) acc[x][y] = mfma_mx4<S>(f.b[x], f.a[y], acc[x][y], w.b[x], w.a[y]);
}

// One slab from stage `cur`; fragments of its first step are in f0, its scales
// in w.  Ends with those of the next slab (stage `nxt`) there.  The loads of the
// slab three ahead go into `prv`, the stage of the slab before, spread over the
// MFMAs (a burst of them would hold up the wave, which issues in order): the
// first kAfter were issued behind the last barrier.
template <class T>
__device__ __forceinline__ void slab(f32x16_t (&acc)[T::FN][T::FM], Frags<T>& f0, ScaleWords<T>& w,
                                     typename T::Stage& prv, typename T::Stage& cur, const typename T::Stage& nxt,
                                     const Source& A, const Source& B, int u, int last, int wave, int lane, int ra,
                                     int rb) {
  constexpr int FM = T::FM, FN = T::FN, kMid = T::kAfter + (T::kLoads - T::kAfter) * 2 / 3;
  Frags<T> f1;
  read_frag<FN>(f1.b, cur, rb, lane, 1);
  read_frag<FM>(f1.a, cur, ra, lane, 1);
  load_unit<T, T::kAfter, kMid>(prv, A, B, u + kStages - 1, last, wave, lane);
  mfmas<T, 0, 0, FM>(acc, f0, w);
  if constexpr (FM * FN >= FM + FN) {
#pragma unroll
    for (int g = 0; g < FM + FN; ++g) {
      __builtin_amdgcn_sched_group_barrier(kSchedDsRead, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedMfma, FM * FN / (FM + FN), 0);
      __builtin_amdgcn_sched_group_barrier(kSchedVmem, 1, 0);
    }
  }
  __builtin_amdgcn_sched_barrier(0);
  load_unit<T, kMid, T::kLoads>(prv, A, B, u + kStages - 1, last, wave, lane);
  mfmas<T, 1, 0, FM / 2>(acc, f1, w);
  if constexpr (FM * FN >= FM + FN) {
#pragma unroll
    for (int g = 0; g < T::kLoads - kMid; ++g) {
      __builtin_amdgcn_sched_group_barrier(kSchedMfma, FM * FN / 2 / (T::kLoads - kMid), 0);
      __builtin_amdgcn_sched_group_barrier(kSchedVmem, 1, 0);
    }
  }
  __builtin_amdgcn_sched_barrier(0);
  // this wave's part of the next slab has landed (two slabs stay in flight), and
  // all its reads of this one are done
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(2 * T::kLoads, 0));
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  load_unit<T, 0, T::kAfter>(cur, A, B, u + kStages, last, wave, lane);
  ScaleWords<T> wn;
  read_frag<FN>(f0.b, nxt, rb, lane, 0);
  read_frag<FM>(f0.a, nxt, ra, lane, 0);
  read_scales<FN>(wn.b, nxt, rb, lane);
  read_scales<FM>(wn.a, nxt, ra, lane);
  mfmas<T, 1, FM / 2, FM>(acc, f1, w);
#pragma unroll
  for (int g = 0; g < FM * FN / 2; ++g) {
    __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
    __builtin_amdgcn_sched_group_barrier(kSchedDsRead, (2 * (FM + FN) + FM * FN / 2 - 1) / (FM * FN / 2), 0);
    __builtin_amdgcn_sched_group_barrier(kSchedVmem, (T::kAfter + FM * FN / 2 - 1) / (FM * FN / 2), 0);
  }
  __builtin_amdgcn_sched_barrier(0);
  shift_scales<FN>(wn.b, lane);
  shift_scales<FM>(wn.a, lane);
  w = wn;
}

// Block id -> tile: consecutive ids go to the 8 XCDs in turn, so each XCD gets a
// contiguous range of tiles, and tiles run down columns of 4 tile rows, so that
// the tiles an XCD works on at one time share their rows of A and B in its L2.
__device__ __forceinline__ void tile_of(int id, int total, int tm, int tn, int* outer, int* ti, int* tj) {
  const int q = total >> 3, rest = total & 7, x = id & 7, at = id >> 3;
  int t = x * q + (x < rest ? x : rest) + at;
  const int per = tm * tn;
  *outer = t / per;
  t -= *outer * per;
  constexpr int kGroup = 4;
  const int g = t / (kGroup * tn), first = g * kGroup, h = tm - first < kGroup ? tm - first : kGroup;
  t -= g * kGroup * tn;
  *ti = first + t % h;
  *tj = t / h;
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
// straight from the accumulators: 138 -> 122 us.
template <class T, int DC, bool ADD>
__device__ __forceinline__ void store_tile(void* C, const f32x16_t (&acc)[T::FN][T::FM], uint4* stage, int i, int j,
                                           int m, int n, int lane) {
  constexpr int kSize = DC == kF32 ? 4 : 2, kHeld = ADD || DC == kF32 ? 4 : 2;  // bytes of an element of C, in LDS
  constexpr int kCols = 32 * T::FN, kPitch = kCols * kHeld / 16 + 1;            // uint4 of a row, one against conflicts
  constexpr int kLanes = kCols * kSize / 16, kRows = 64 / kLanes;               // lanes of a row, rows of a store
  static_assert(32 * kPitch * 16 <= sizeof(typename T::Stage) && kLanes <= 64, "staging");
  const int row = lane & 31, half = lane >> 5, r0 = lane / kLanes, chunk = lane % kLanes;
  constexpr int kElems = 16 / kSize;
  const int jc = j + chunk * kElems;
#pragma unroll
  for (int y = 0; y < T::FM; ++y) {
#pragma unroll
    for (int x = 0; x < T::FN; ++x)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float v[4] = {acc[x][y][4 * g], acc[x][y][4 * g + 1], acc[x][y][4 * g + 2], acc[x][y][4 * g + 3]};
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
      if (ir < m && jc < n) {
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
        if (jc + kElems <= n) {
          if constexpr (kHeld == 4) {
            if constexpr (ADD) {
              const u32x4_t c = *reinterpret_cast<const u32x4_a2*>(p);
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

template <class T, int DC>
__global__ __launch_bounds__(256, T::TM == 256 ? 1 : 2) void mx4_tile_gemm_kernel(Mx4GemmArgs a, int tm, int tn) {
  typedef typename T::Stage Stage;
  constexpr int FM = T::FM, FN = T::FN;
  __shared__ Stage s0, s1, s2, s3;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)), lane = threadIdx.x & 63;
  int outer, ti, tj;
  tile_of(blockIdx.x, gridDim.x, tm, tn, &outer, &ti, &tj);
  const int b = outer / a.pieces, piece = outer - b * a.pieces;
  const int i0 = ti * T::TM, j0 = tj * T::TN;
  const int ub = piece * a.piece_units, ue = ub + a.piece_units < a.units ? ub + a.piece_units : a.units;
  // lane l fills slot l % 4 of row l / 4 of each 16-row piece
  const int vcode = (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 4) & 3)) * 16);
  const int fa = i0 + wave * (T::TM / 4), fb = j0 + wave * (T::TN / 4);  // first rows of this wave's loads
  const Source A{a.A[b], a.As[b], fa * 64 + vcode, (fa + lane) * 4, static_cast<uint32_t>(a.m),
                 static_cast<uint32_t>(a.units) * a.m};
  const Source B{a.B[b], a.Bs[b], fb * 64 + vcode, (fb + lane) * 4, static_cast<uint32_t>(a.n),
                 static_cast<uint32_t>(a.units) * a.n};
  const int last = a.units - 1;
  Stage* st[kStages] = {&s0, &s1, &s2, &s3};
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) load_unit<T, 0, T::kLoads>(*st[s], A, B, ub + s, last, wave, lane);
  load_unit<T, 0, T::kAfter>(s3, A, B, ub + 3, last, wave, lane);
  const int ra = FM * 32 * (wave / T::WN), rb = T::TM + FN * 32 * (wave % T::WN);
  f32x16_t acc[FN][FM] = {};
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(2 * T::kLoads + T::kAfter, 0));
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  Frags<T> f;
  ScaleWords<T> w;
  read_frag<FN>(f.b, s0, rb, lane, 0);
  read_frag<FM>(f.a, s0, ra, lane, 0);
  read_scales<FN>(w.b, s0, rb, lane);
  read_scales<FM>(w.a, s0, ra, lane);
  shift_scales<FN>(w.b, lane);
  shift_scales<FM>(w.a, lane);
  int u = ub;
  for (; u + kStages <= ue; u += kStages) {
    slab<T>(acc, f, w, s3, s0, s1, A, B, u, last, wave, lane, ra, rb);
    slab<T>(acc, f, w, s0, s1, s2, A, B, u + 1, last, wave, lane, ra, rb);
    slab<T>(acc, f, w, s1, s2, s3, A, B, u + 2, last, wave, lane, ra, rb);
    slab<T>(acc, f, w, s2, s3, s0, A, B, u + 3, last, wave, lane, ra, rb);
  }
  if (u < ue) slab<T>(acc, f, w, s3, s0, s1, A, B, u, last, wave, lane, ra, rb);
  if (u + 1 < ue) slab<T>(acc, f, w, s0, s1, s2, A, B, u + 1, last, wave, lane, ra, rb);
  if (u + 2 < ue) slab<T>(acc, f, w, s1, s2, s3, A, B, u + 2, last, wave, lane, ra, rb);
  // loads behind the last unit are still on their way into LDS: they end here,
  // and so do all waves' reads, before LDS takes the results
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
  asm volatile("s_barrier" ::: "memory");
  const int i = i0 + ra, j = j0 + rb - T::TM;  // this wave's first row and column
  uint4* const stage = wave == 0 ? s0.code : wave == 1 ? s1.code : wave == 2 ? s2.code : s3.code;
  if (a.pieces > 1) {
    float* part = a.partial + (static_cast<int64_t>(piece) * a.batch + b) * a.m * a.n;
    store_tile<T, kF32, false>(part, acc, stage, i, j, a.m, a.n, lane);
  } else if (a.accumulate) {
    store_tile<T, DC, true>(a.C[b], acc, stage, i, j, a.m, a.n, lane);
  } else {
    store_tile<T, DC, false>(a.C[b], acc, stage, i, j, a.m, a.n, lane);
  }
}

// ---------------------------------------------------------------------------
// The pieces of a product that was split along k, added in their order.
// ---------------------------------------------------------------------------
template <int DC>
__global__ __launch_bounds__(256) void mx4_join_kernel(Mx4GemmArgs a) {
  const int b = blockIdx.z;
  const int64_t mn = static_cast<int64_t>(a.m) * a.n, step = static_cast<int64_t>(a.batch) * mn;
  const float* part = a.partial + b * mn;
  void* C = a.C[b];
  const bool vec = (mn & 3) == 0 && (reinterpret_cast<uintptr_t>(C) & (DC == kF32 ? 15u : 7u)) == 0;
  for (int64_t at = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4; at < mn;
       at += static_cast<int64_t>(gridDim.x) * 1024) {
    const int left = mn - at < 4 ? static_cast<int>(mn - at) : 4;
    float v[4] = {};
    for (int p = 0; p < a.pieces; ++p) {
      if (vec) {
        const float4 x = *reinterpret_cast<const float4*>(part + p * step + at);
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < left) v[e] += part[p * step + at + e];
      }
    }
    store_quad<DC>(C, at, v, left, vec, a.accumulate);
  }
}

// ---------------------------------------------------------------------------
// At most 16 rows of A (a few tokens against a weight): the codes of B are what
// has to be read.  A wave takes NT tiles of 16 rows of B (v_mfma_scale_f32_
// 16x16x128_f8f6f4: a lane holds one block of one row, a unit of 16 rows is 1 KB
// of contiguous memory) and every NW-th unit of k, straight from memory into
// registers; the block's NW sums are added in LDS, in their order.  Rows of A
// behind the last one repeat it and are not stored.
// ---------------------------------------------------------------------------
constexpr int kFewRows = 16;
constexpr int kUnitsAhead = 2;

template <int NT, int NW, int DC>
__global__ __launch_bounds__(64 * NW) void mx4_few_rows_kernel(Mx4GemmArgs a) {
  __shared__ f32x4_t sums[NW][NT][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, b = blockIdx.z;
  const int j0 = blockIdx.x * 16 * NT, r = lane & 15, blk = lane >> 4;
  const uint4* A = static_cast<const uint4*>(a.A[b]) + blk;
  const uint4* B = static_cast<const uint4*>(a.B[b]) + blk;
  const uint8_t* As = static_cast<const uint8_t*>(a.As[b]) + blk;
  const uint8_t* Bs = static_cast<const uint8_t*>(a.Bs[b]) + blk;
  const int ra = r < a.m ? r : a.m - 1;
  int rb[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) rb[t] = j0 + 16 * t + r < a.n ? j0 + 16 * t + r : a.n - 1;
  f32x4_t acc[NT] = {};
  for (int u0 = wave; u0 < a.units; u0 += NW * kUnitsAhead) {
    uint4 av[kUnitsAhead], bv[kUnitsAhead][NT];
    uint32_t sa[kUnitsAhead], sb[kUnitsAhead][NT];
#pragma unroll
    for (int k = 0; k < kUnitsAhead; ++k) {
      const int u = u0 + k * NW;
      const bool in = u < a.units;  // a unit behind the last one counts as zeros
      const int64_t la = static_cast<int64_t>(in ? u : u0) * a.m + ra;
      av[k] = A[la * 4];
      sa[k] = As[la * 4];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int64_t lb = static_cast<int64_t>(in ? u : u0) * a.n + rb[t];
        bv[k][t] = B[lb * 4];
        sb[k][t] = Bs[lb * 4];
      }
    }
#pragma unroll
    for (int k = 0; k < kUnitsAhead; ++k) {
      if (u0 + k * NW < a.units) {
        const i32x8_t x = {static_cast<int>(av[k].x), static_cast<int>(av[k].y), static_cast<int>(av[k].z),
                           static_cast<int>(av[k].w), 0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const i32x8_t y = {static_cast<int>(bv[k][t].x), static_cast<int>(bv[k][t].y), static_cast<int>(bv[k][t].z),
                             static_cast<int>(bv[k][t].w), 0, 0, 0, 0};
          acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(y, x, acc[t], kFp4, kFp4, 0,
                                                                    static_cast<int>(sb[k][t]), 0,
                                                                    static_cast<int>(sa[k]));
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) sums[wave][t][lane] = acc[t];
  __syncthreads();
  // lane l of a tile: row l % 16 of C, columns 4 (l / 16) .. + 3
  void* C = a.C[b];
  const bool vec = (a.n & 3) == 0 && (reinterpret_cast<uintptr_t>(C) & (DC == kF32 ? 15u : 7u)) == 0;
  for (int p = threadIdx.x; p < 64 * NT; p += 64 * NW) {
    const int t = p >> 6, l = p & 63, i = l & 15, j = j0 + 16 * t + 4 * (l >> 4);
    if (i >= a.m || j >= a.n) continue;
    f32x4_t s = sums[0][t][l];
#pragma unroll
    for (int q = 1; q < NW; ++q) s += sums[q][t][l];
    const float v[4] = {s[0], s[1], s[2], s[3]};
    store_quad<DC>(C, static_cast<int64_t>(i) * a.n + j, v, a.n - j, vec, a.accumulate);
  }
}

typedef Tile<256, 256, 2> Big;
typedef Tile<128, 128, 2> Mid;
typedef Tile<64, 128, 1> Low;

int ceil_div(int a, int b) { return (a + b - 1) / b; }

template <class T>
int64_t tiles_of(int batch, int m, int n) {
  return static_cast<int64_t>(ceil_div(m, T::TM)) * ceil_div(n, T::TN) * batch;
}

// Pieces along k of a product in 64 x 128 tiles that leave compute units idle:
// the fewest microseconds of a slab a unit (measured 0.26, one block on a compute
// unit) plus, for more than one piece, the joining launch (4.5) and the partial
// sums' way through memory (8 bytes an element and piece at 6 TB/s).
void split_k(int64_t tiles, int units, double elements, Mx4Plan* p) {
  constexpr int kMinUnits = 4;  // of a piece
  double best = 0.0;
  for (int q = 1; q * tiles <= kCUs && (q == 1 || units / q >= kMinUnits); ++q) {
    const double us = ceil_div(units, q) * 0.26 + (q > 1 ? 4.5 + q * elements * 8.0 / 6e6 : 0.0);
    if (q == 1 || us < best) {
      best = us;
      p->piece_units = ceil_div(units, q);
      p->pieces = ceil_div(units, p->piece_units);
    }
  }
}

}  // namespace

// Which kernel, by the tiles there are for 256 compute units (times on bf16 C):
//   at most 16 rows of A   B's codes are read once, straight into registers.
//                          16x18944x3584: 9.3 us, 64 x 128 tiles 10.2
//   256 x 256 tiles        where their rounds together leave at most a third of the
//                          compute units idle: 4096x4096x2048 (256 tiles) 25.9 us,
//                          128 x 128 28.3; 2048x4096x8192 (128 tiles) 46.9 and 42.1.
//                          From 513 tiles on that is always so, however few the last
//                          round has.  At k = 8192 it is right at every count
//                          measured (256 x 256 / 128 x 128): 171 tiles 48.8 / 56.8,
//                          342 100 / 106, 520 156 / 163, 780 214 / 235, and 300, which
//                          it leaves, 98.3 / 94.1.  At k = 2048 a tile's start and end
//                          weigh more and the smaller tiles would win behind a full
//                          round: 171 21.4 / 20.8, 342 39.9 / 35.1, 520 62.1 / 52.6,
//                          780 82.9 / 77.6, but 512 (two full ones) 46.3 / 49.6.
//   64 x 128 tiles         for at most 384 of them, split along k if they are
//                          few: 512x3584x3584 (224) 9.6 us, 128 x 128 11.4;
//                          256x18944x3584 (592) 22.0 and 19.0
//   128 x 128 tiles        otherwise.
Mx4Plan mx4_plan(int batch, int m, int n, int k) {
  const int units = static_cast<int>(mx4_units(k));
  Mx4Plan p{kMxFewRows, 1, units, 0};
  if (m <= kFewRows) return p;
  const int64_t big = tiles_of<Big>(batch, m, n), low = tiles_of<Low>(batch, m, n);
  const int64_t rounds = (big + kCUs - 1) / kCUs;
  if (big * 3 >= rounds * kCUs * 2) {
    p.kind = kMxBig;
  } else if (low * 2 <= kCUs * 3) {
    p.kind = kMxLow;
    const double elements = static_cast<double>(batch) * m * n;
    split_k(low, units, elements, &p);
    if (p.pieces > 1) p.bytes = static_cast<size_t>(p.pieces) * batch * m * n * sizeof(float);
  } else {
    p.kind = kMxMid;
  }
  return p;
}

template <class T>
static void launch_tiles(const Mx4GemmArgs& a, hipStream_t s) {
  const int tm = ceil_div(a.m, T::TM), tn = ceil_div(a.n, T::TN);
  const dim3 grid(static_cast<uint32_t>(tm) * tn * a.batch * a.pieces), block(256);
  if (a.c_dtype == kF32) {
    hipLaunchKernelGGL((mx4_tile_gemm_kernel<T, kF32>), grid, block, 0, s, a, tm, tn);
  } else {
    hipLaunchKernelGGL((mx4_tile_gemm_kernel<T, kBF16>), grid, block, 0, s, a, tm, tn);
  }
}

template <int NT, int NW>
static void launch_few(const Mx4GemmArgs& a, hipStream_t s) {
  const dim3 grid(ceil_div(a.n, 16 * NT), 1, a.batch), block(64 * NW);
  if (a.c_dtype == kF32) {
    hipLaunchKernelGGL((mx4_few_rows_kernel<NT, NW, kF32>), grid, block, 0, s, a);
  } else {
    hipLaunchKernelGGL((mx4_few_rows_kernel<NT, NW, kBF16>), grid, block, 0, s, a);
  }
}

hipError_t launch_mx4_gemm(const Mx4GemmArgs& a, Mx4Kind kind, hipStream_t s) {
  switch (kind) {
    case kMxBig: launch_tiles<Big>(a, s); break;
    case kMxMid: launch_tiles<Mid>(a, s); break;
    case kMxLow: launch_tiles<Low>(a, s); break;
    default:
      // 16 waves a block where 8 leave compute units idle or with few loads in
      // flight and k is long: 1x3584x18944 10.1 -> 8.0 us, 1x18944x3584 8.2 -> 9.3
      if (a.units >= 64 && ceil_div(a.n, 16) * a.batch <= kCUs) {
        launch_few<1, 16>(a, s);
      } else {
        launch_few<1, 8>(a, s);
      }
      break;
  }
  return hipGetLastError();
}

hipError_t launch_mx4_join(const Mx4GemmArgs& a, hipStream_t s) {
  const int64_t blocks = (static_cast<int64_t>(a.m) * a.n + 1023) / 1024;
  const dim3 grid(static_cast<uint32_t>(blocks < 4096 ? blocks : 4096), 1, a.batch), block(256);
  if (a.c_dtype == kF32) {
    hipLaunchKernelGGL(mx4_join_kernel<kF32>, grid, block, 0, s, a);
  } else {
    hipLaunchKernelGGL(mx4_join_kernel<kBF16>, grid, block, 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace muon

// The tile kernel of the products of 8-bit codes, in two ways of multiplying:
//
// kFast, for bf16 results: the block-scaled MFMA with fp8 operands (32x32x64: a lane
// holds 32 bytes of one row and their scale byte, a power of two that the MFMA
// applies).  It adds eight neighbouring products at a time with 13 bits below the
// largest of them (measured: 1 beside 2^13 counts, beside 2^14 it is lost), and those
// sums to the fp32 accumulator: 2^-16 of a normal sum, 1/100 of bf16's rounding.
// From registers alone it reaches 3800 TFLOP/s here.
//
// kExact, for fp32 results: codes times their scales are bf16 numbers (exactly, down
// to 2^-133), so v_cvt_scalef32_pk_bf16_{fp8,bf8} makes operands of the bf16 MFMA
// (32x32x16) whose products and sums are fp32's: 2^-26 of a normal sum.  1700
// TFLOP/s from registers, conversions (in the MFMAs' shadow) included 1670.
//
// TM x TN tiles by 4 waves (WM x 4 / WM, each FM x FN MFMA tiles).  k runs in slabs
// of 64, half a unit: the tile's codes (each operand one contiguous run of memory)
// go straight into a ring of 4 LDS stages, and with the first slab of a unit its
// scales.  The order of k is free as long as A and B agree: lanes 0..31 take the
// first 32 bytes of their row, lanes 32..63 the others.  Chunk b of row r lies in
// slot b ^ (r / 4 % 4) of the row's 64 bytes, so that 16 lanes reading one chunk of
// 16 rows touch all LDS banks once; the permutation is in the global addresses of
// the loads, which stay within a row's 64 bytes.
//
// A slab's fragments are read into registers while the MFMAs of the slab before
// run, so that behind the one barrier of a slab its stage can be filled anew.
#pragma once

#include "muon_fp8.h"
#include "muon_tile.h"

namespace muon {
namespace fp8 {

constexpr int kStages = 4;
constexpr bool kFast = false, kExact = true;

template <int TM_, int TN_, int WM_>
struct Tile {
  static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = 4 / WM_;
  static constexpr int FM = TM / WM / 32, FN = TN / WN / 32;
  static constexpr int kCodeLoads = TM / 64 + TN / 64;  // per wave and slab
  struct Stage {
    uint4 code[(TM + TN) * 4];  // A rows, then B rows, 4 slots each
  };
};

// A unit's scales of A and of B, from a multiple of 16 rows on: what one load of a
// wave fills, though the rows of a tile are at most 17 of its 64 lanes' 16 bytes.
struct ScaleStage {
  uint8_t a[1024], b[1024];
};

// One operand's source (block-uniform but for vcode).
struct Source {
  const void* code;
  int vcode;       // byte offset of this lane's first load from a piece's first row
  uint32_t rows;
};
// What this wave loads of the scales, A's or B's.
struct ScaleSource {
  const void* scale;
  int voff;        // byte offset of this lane's load from a unit's first row, or behind everything
  uint32_t pitch;
};

__device__ __forceinline__ uint32_t clip(uint64_t bytes) { return bytes < 0x7fffffffu ? static_cast<uint32_t>(bytes) : 0x7fffffffu; }

// The loads that bring this wave's share of slab s into a stage: the codes of A and
// of B, 16 rows each.  Behind the last slab the last one is read again.  The
// resource starts at the piece and ends with the matrix, so every load is checked
// against the matrix's end: rows behind the last row read the next piece's, or
// zeros behind the last piece.  Neither enters a stored element.
template <class T>
__device__ __forceinline__ void load_slab(typename T::Stage& st, const Source& A, const Source& B, int s, int slabs,
                                          int wave) {
  constexpr int RA = T::TM / 4, RB = T::TN / 4;  // rows of this wave
  const uint32_t p = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(s < slabs ? s : slabs - 1));
  const uint64_t la = static_cast<uint64_t>(p) * A.rows, lb = static_cast<uint64_t>(p) * B.rows;
  const __amdgpu_buffer_rsrc_t ca = make_rsrc(A.code, la * 64, clip((static_cast<uint64_t>(slabs) * A.rows - la) * 64));
  const __amdgpu_buffer_rsrc_t cb = make_rsrc(B.code, lb * 64, clip((static_cast<uint64_t>(slabs) * B.rows - lb) * 64));
  lds_ptr_t da = (lds_ptr_t)(st.code + wave * RA * 4), db = (lds_ptr_t)(st.code + (T::TM + wave * RB) * 4);
#define FP8_LOAD(R, RSRC, DST, VOFF, PIECE)     \
  if constexpr ((PIECE) * 1024 < (R) * 64)      \
    __builtin_amdgcn_raw_ptr_buffer_load_lds(RSRC, DST, 16, VOFF, 0, (PIECE) * 1024, 0)
  FP8_LOAD(RA, ca, da, A.vcode, 0);
  FP8_LOAD(RA, ca, da, A.vcode, 1);
  FP8_LOAD(RA, ca, da, A.vcode, 2);
  FP8_LOAD(RA, ca, da, A.vcode, 3);
  FP8_LOAD(RB, cb, db, B.vcode, 0);
  FP8_LOAD(RB, cb, db, B.vcode, 1);
  FP8_LOAD(RB, cb, db, B.vcode, 2);
  FP8_LOAD(RB, cb, db, B.vcode, 3);
#undef FP8_LOAD
  static_assert(RA % 16 == 0 && RB % 16 == 0 && RA <= 64 && RB <= 64, "loads of a slab");
}

// One load: even waves bring A's scales of the unit that slab s begins, odd ones B's,
// two of them the same bytes, so that every wave has the same loads under way.
// Lanes behind the tile's rows have an offset behind the matrix and write zeros.
__device__ __forceinline__ void load_scales(ScaleStage& st, const ScaleSource& S, int s, int slabs, int wave) {
  const uint32_t p = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(s < slabs ? s : slabs - 1));
  const uint64_t at = static_cast<uint64_t>(p >> 1) * S.pitch;
  const __amdgpu_buffer_rsrc_t r = make_rsrc(S.scale, at, clip(static_cast<uint64_t>(slabs >> 1) * S.pitch - at));
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)((wave & 1) != 0 ? st.b : st.a), 16, S.voff, 0, 0, 0);
}

struct Frag {
  uint4 lo, hi;
};
template <class T>
struct Frags {
  Frag a[T::FM], b[T::FN];
};
template <class T>
struct Scales {
  uint32_t a[T::FM], b[T::FN];
};

// The 32-row fragments from row `first` of a stage on.
template <int F, class Stage>
__device__ __forceinline__ void read_frag(Frag (&f)[F], const Stage& st, int first, int lane) {
  const int r = lane & 31, swap = (r >> 2) & 3, at = 2 * (lane >> 5);
#pragma unroll
  for (int x = 0; x < F; ++x) {
    f[x].lo = st.code[(first + 32 * x + r) * 4 + (at ^ swap)];
    f[x].hi = st.code[(first + 32 * x + r) * 4 + ((at + 1) ^ swap)];
  }
}
template <int F>
__device__ __forceinline__ void read_scales(uint32_t (&w)[F], const uint8_t* scale, int first, int lane) {
#pragma unroll
  for (int x = 0; x < F; ++x) w[x] = scale[first + 32 * x + (lane & 31)];
}

__device__ __forceinline__ i32x8_t operand(const Frag& f) {
  return (i32x8_t){static_cast<int>(f.lo.x), static_cast<int>(f.lo.y), static_cast<int>(f.lo.z), static_cast<int>(f.lo.w),
                   static_cast<int>(f.hi.x), static_cast<int>(f.hi.y), static_cast<int>(f.hi.z), static_cast<int>(f.hi.w)};
}

template <class T, int FA>
__device__ __forceinline__ void mfmas(f32x16_t (&acc)[T::FN][T::FM], const Frags<T>& f, const Scales<T>& w) {
#pragma unroll
  for (int y = 0; y < T::FM; ++y)
#pragma unroll
    for (int x = 0; x < T::FN; ++x)
      acc[x][y] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(f.b[x]), operand(f.a[y]), acc[x][y], kE4M3, FA, 0,
                                                                  static_cast<int>(w.b[x]), 0, static_cast<int>(w.a[y]));
}

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

// Bytes 8 s .. 8 s + 7 of a fragment times their scale, as bf16.
template <int F, int S>
__device__ __forceinline__ bf16x8_t to_bf16(const Frag& f, uint32_t byte) {
  const float scale = __uint_as_float(byte << 23);
  const uint4 q = S < 2 ? f.lo : f.hi;
  const uint32_t lo = S % 2 == 0 ? q.x : q.z, hi = S % 2 == 0 ? q.y : q.w;
  bf16x2_t p0, p1, p2, p3;
  if constexpr (F == kE4M3) {
    p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  } else {
    p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, scale, false);
    p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, scale, true);
    p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, scale, false);
    p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, scale, true);
  }
  return (bf16x8_t){p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// The operands of one of a slab's four steps of 16.
template <class T>
struct Wide {
  bf16x8_t a[T::FM], b[T::FN];
};
template <class T, int FA, int S>
__device__ __forceinline__ void widen(Wide<T>& v, const Frags<T>& f, const Scales<T>& w) {
#pragma unroll
  for (int x = 0; x < T::FN; ++x) v.b[x] = to_bf16<kE4M3, S>(f.b[x], w.b[x]);
#pragma unroll
  for (int y = 0; y < T::FM; ++y) v.a[y] = to_bf16<FA, S>(f.a[y], w.a[y]);
}
template <class T>
__device__ __forceinline__ void mfmas(f32x16_t (&acc)[T::FN][T::FM], const Wide<T>& v) {
#pragma unroll
  for (int y = 0; y < T::FM; ++y)
#pragma unroll
    for (int x = 0; x < T::FN; ++x)
      acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v.b[x], v.a[y], acc[x][y], 0, 0, 0);
}

// Where a wave reads in a stage.
struct Reads {
  int a, b;    // first rows of its fragments
  int sa, sb;  // first scales
};

// One slab from stage `cur`, whose fragments are in f and scales in w; leaves those
// of the next slab (stage `nxt`) there.  The loads of the slab 4 ahead go into `cur`
// and, in even slabs, those of the scales of the unit two ahead into `sc`; odd slabs
// read the next unit's scales from `sc`.  Loads and reads are spread over the MFMAs
// (a burst of them would hold up the wave, which issues in order).
template <class T, int FA, bool EXACT, bool ODD>
__device__ __forceinline__ void slab(f32x16_t (&acc)[T::FN][T::FM], Frags<T>& f, Scales<T>& w, Wide<T>& v,
                                     typename T::Stage& cur, const typename T::Stage& nxt, ScaleStage& sc, const Source& A,
                                     const Source& B, const ScaleSource& S, int s, int slabs, int wave, int lane,
                                     const Reads& at) {
  constexpr int M = T::FM * T::FN, kLoads = T::kCodeLoads + (ODD ? 0 : 1);
  constexpr int kReads = (ODD ? 3 : 2) * (T::FM + T::FN);
  // this wave's part of the next slab has landed (two slabs stay under way), and all
  // its reads of this one are done
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(2 * T::kCodeLoads + 1, 0));
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  Frags<T> fn;
  Scales<T> wn;
  load_slab<T>(cur, A, B, s + kStages, slabs, wave);
  if constexpr (!ODD) load_scales(sc, S, s + kStages, slabs, wave);
  read_frag<T::FN>(fn.b, nxt, at.b, lane);
  read_frag<T::FM>(fn.a, nxt, at.a, lane);
  if constexpr (ODD) {
    read_scales<T::FN>(wn.b, sc.b, at.sb, lane);
    read_scales<T::FM>(wn.a, sc.a, at.sa, lane);
  }
  if constexpr (!EXACT) {
    mfmas<T, FA>(acc, f, w);
#pragma unroll
    for (int g = 0; g < M; ++g) {
      __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedDsRead, (2 * kReads + M - 1) / M, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedVmem, (kLoads + M - 1) / M, 0);
    }
  } else {
    // operands of a step are made while the MFMAs of the step before run
    constexpr int kMake = 4 * (T::FM + T::FN);
    Wide<T> v1;
    mfmas<T>(acc, v);
    widen<T, FA, 1>(v1, f, w);
    mfmas<T>(acc, v1);
    widen<T, FA, 2>(v, f, w);
#pragma unroll
    for (int g = 0; g < 2 * M; ++g) {
      __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedValu, (kMake + M - 1) / M, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedDsRead, (kReads + M - 1) / M, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedVmem, (kLoads + M - 1) / M, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    mfmas<T>(acc, v);
    widen<T, FA, 3>(v1, f, w);
    mfmas<T>(acc, v1);
    widen<T, FA, 0>(v, fn, ODD ? wn : w);
#pragma unroll
    for (int g = 0; g < 2 * M; ++g) {
      __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedValu, (kMake + M - 1) / M, 0);
    }
  }
  __builtin_amdgcn_sched_barrier(0);
  f = fn;
  if constexpr (ODD) w = wn;
}

template <class T>
struct Lds {
  typename T::Stage &s0, &s1, &s2, &s3;
  ScaleStage &c0, &c1;
};

// Units ub .. ue - 1 of the tile at rows i0 of A and j0 of B into the accumulators.
// All of the block's LDS is free behind it.  (The stages are objects of their own so
// that the compiler can tell a read of one from a load into another.)
template <class T, int FA, bool EXACT>
__device__ __forceinline__ void tile_product(f32x16_t (&acc)[T::FN][T::FM], const Lds<T>& lds, Source A, Source B,
                                             const void* a_scale, const void* b_scale, int i0, int j0, int ub, int ue,
                                             int units, int wave, int lane) {
  // lane l fills slot l % 4 of row l / 4 of each 16-row run
  const int vcode = (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 4) & 3)) * 16);
  A.vcode = (i0 + wave * (T::TM / 4)) * 64 + vcode;
  B.vcode = (j0 + wave * (T::TN / 4)) * 64 + vcode;
  const bool odd = (wave & 1) != 0;
  const int lines = (odd ? T::TN : T::TM) / kF8Line + 1;
  const uint32_t rows = odd ? B.rows : A.rows;
  const ScaleSource S{odd ? b_scale : a_scale, lane < lines ? ((odd ? j0 : i0) & ~(kF8Line - 1)) + lane * 16 : 0x7ffffff0,
                      (rows + kF8Line - 1) & ~(kF8Line - 1u)};
  const int ra = T::FM * 32 * (wave / T::WN), rb = T::FN * 32 * (wave % T::WN);
  const Reads at{ra, T::TM + rb, (i0 & (kF8Line - 1)) + ra, (j0 & (kF8Line - 1)) + rb};
  const int slabs = 2 * units, se = 2 * ue;
  int s = 2 * ub;
  load_slab<T>(lds.s0, A, B, s, slabs, wave);
  load_scales(lds.c0, S, s, slabs, wave);
  load_slab<T>(lds.s1, A, B, s + 1, slabs, wave);
  load_slab<T>(lds.s2, A, B, s + 2, slabs, wave);
  load_scales(lds.c1, S, s + 2, slabs, wave);
  load_slab<T>(lds.s3, A, B, s + 3, slabs, wave);
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(3 * T::kCodeLoads + 1, 0));  // the first slab has landed
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  Frags<T> f;
  Scales<T> w;
  read_frag<T::FN>(f.b, lds.s0, at.b, lane);
  read_frag<T::FM>(f.a, lds.s0, at.a, lane);
  read_scales<T::FN>(w.b, lds.c0.b, at.sb, lane);
  read_scales<T::FM>(w.a, lds.c0.a, at.sa, lane);
  Wide<T> v;
  if constexpr (EXACT) widen<T, FA, 0>(v, f, w);
  for (; s + kStages <= se; s += kStages) {
    slab<T, FA, EXACT, false>(acc, f, w, v, lds.s0, lds.s1, lds.c0, A, B, S, s, slabs, wave, lane, at);
    slab<T, FA, EXACT, true>(acc, f, w, v, lds.s1, lds.s2, lds.c1, A, B, S, s + 1, slabs, wave, lane, at);
    slab<T, FA, EXACT, false>(acc, f, w, v, lds.s2, lds.s3, lds.c1, A, B, S, s + 2, slabs, wave, lane, at);
    slab<T, FA, EXACT, true>(acc, f, w, v, lds.s3, lds.s0, lds.c0, A, B, S, s + 3, slabs, wave, lane, at);
  }
  if (s < se) {
    slab<T, FA, EXACT, false>(acc, f, w, v, lds.s0, lds.s1, lds.c0, A, B, S, s, slabs, wave, lane, at);
    slab<T, FA, EXACT, true>(acc, f, w, v, lds.s1, lds.s2, lds.c1, A, B, S, s + 1, slabs, wave, lane, at);
  }
  // loads behind the last unit are still on their way into LDS: they end here, and
  // so do all waves' reads
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
  asm volatile("s_barrier" ::: "memory");
}

// A wave's accumulators to C (rows under m, columns under n); fp32 C for exact sums.
template <class T, bool EXACT>
__device__ __forceinline__ void store_product(void* C, const f32x16_t (&acc)[T::FN][T::FM], typename T::Stage& stage, int i,
                                              int j, int m, int n, int lane, int accumulate) {
  constexpr int DC = EXACT ? kF32 : kBF16;
  if (accumulate) {
    store_tile<T, DC, true>(C, acc, stage.code, i, j, m, n, lane);
  } else {
    store_tile<T, DC, false>(C, acc, stage.code, i, j, m, n, lane);
  }
}

typedef Tile<256, 256, 2> Big;
typedef Tile<128, 128, 2> Mid;
typedef Tile<64, 128, 1> Low;

// The block's LDS, `lds`.
#define FP8_LDS(T)                                  \
  __shared__ typename T::Stage s0, s1, s2, s3;      \
  __shared__ ScaleStage c0, c1;                     \
  const Lds<T> lds{s0, s1, s2, s3, c0, c1}

template <class T>
constexpr int kBlocksPerCU = T::TM == 256 ? 1 : 2;

}  // namespace fp8
}  // namespace muon

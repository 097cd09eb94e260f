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
//
// 256 x 256 tiles are bound by power: 4096 x 4096 x 18944 of normal numbers 216 us, 2.94
// PFLOP/s, of zeros 158 us, 4.02 (another time 238 and 165).  8192 x 8192 x 8192 394 us,
// 2.79 PFLOP/s, with fp32 results 756 us, 1.45.  128 x 128 tiles, two blocks a compute unit,
// read LDS for half as many products: 2048 x 4096 x 8192 59 us, 2.34 PFLOP/s.  64 x 128 tiles
// wait for loads and barriers, 0.33 us a unit (fp32 results 0.55).  The kernels of 256 x 256
// tiles with bf16 results spill 32 to 48 registers, the one whose blocks stay 11, none of
// them within the loop over slabs.
//
// Times beside the rules that choose between tiles: medians of 7 turns of 20 calls, the
// sides in turn on one card (turns within 3 % of each other).  In one row of calls a kernel
// that is bound by power starts as fast, is up to a quarter slower about the tenth to the
// twentieth call, and settles between: 16380 rows over 64 experts 265, 360, then 300 us.
//
// Blocks that fill a compute unit can stay for tile after tile: what they load runs 4
// slabs ahead of what they multiply, over the end of a tile into the next one, whose
// first slabs are there when a tile's results have gone.  A tile takes whole rounds of
// the ring: behind an odd number of units two slabs are loaded for nothing.  That pays
// where k is short against the results: the weight gradients of 16 experts of 2048 x
// 7168 with 8190 rows in all take 334 us so and 350 with a block a tile (with as many rows
// for every expert 296 and 356).  Long products are limited by power and gain nothing
// (8192x8192x8192 bf16 389 and 391 us).
#pragma once

#include <cmath>
#include <type_traits>

#include "muon_fp8.h"
#include "muon_tile.h"

namespace muon {
namespace fp8 {

constexpr bool kFast = false, kExact = true;

template <int TM_, int TN_, int WM_, bool STAYS = false>
struct Tile {
  static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = 4 / WM_;
  static constexpr int FM = TM / WM / 32, FN = TN / WN / 32;
  static constexpr int kCodeLoads = TM / 64 + TN / 64;  // per wave and slab
  static constexpr bool kStays = STAYS;                 // its block takes tile after tile
  static constexpr int kStores = FM * FN * 4;           // of a wave and tile of fp32 results, 1 KB each
  struct Stage {
    uint4 code[(TM + TN) * 4];  // A rows, then B rows, 4 slots each
  };
};

// A unit's scales of A and of B, from a multiple of 16 rows on: what one load of a
// wave fills, though the rows of a tile are at most 17 of its 64 lanes' 16 bytes.
struct ScaleStage {
  uint8_t a[1024], b[1024];
};

__device__ __forceinline__ uint32_t clip(uint64_t bytes) {
  return (bytes >> 31) != 0 ? 0x7fffffffu : static_cast<uint32_t>(bytes);
}

// One operand of a tile (block-uniform): codes and scales of its matrix, its first
// row, and the matrix's rows and units.
struct Operand {
  const void* code;
  const void* scale;
  int row;
  uint32_t rows;
  int units;
};

// What is loaded next (block-uniform): addresses of the tile's first row in the next
// slab, for the scales of the operand that this wave brings them of, and the bytes
// from there to the end of the matrix, which every load is checked against: rows
// behind the last row read the next piece's, or zeros behind the last piece.
// Neither enters a stored element.
struct Stream {
  uint64_t a, b, s;
  uint64_t a_left, b_left, s_left;
  uint32_t a_step, b_step, s_step;
  int slabs;  // of the tile, still to load

  // Units ub .. ue - 1 (at least one) of a tile.
  __device__ __forceinline__ void start(const Operand& A, const Operand& B, int ub, int ue, int wave) {
    a_step = A.rows * kF8Piece;
    b_step = B.rows * kF8Piece;
    const uint64_t at_a = 2 * static_cast<uint64_t>(ub) * a_step + static_cast<uint64_t>(A.row) * kF8Piece;
    const uint64_t at_b = 2 * static_cast<uint64_t>(ub) * b_step + static_cast<uint64_t>(B.row) * kF8Piece;
    a = reinterpret_cast<uint64_t>(A.code) + at_a;
    b = reinterpret_cast<uint64_t>(B.code) + at_b;
    a_left = 2 * static_cast<uint64_t>(A.units) * a_step - at_a;
    b_left = 2 * static_cast<uint64_t>(B.units) * b_step - at_b;
    const bool of_b = (wave & 1) != 0;
    s_step = ((of_b ? B.rows : A.rows) + kF8Line - 1) & ~(kF8Line - 1u);
    const uint64_t at_s = static_cast<uint64_t>(ub) * s_step + ((of_b ? B.row : A.row) & ~(kF8Line - 1));
    s = (of_b ? reinterpret_cast<uint64_t>(B.scale) : reinterpret_cast<uint64_t>(A.scale)) + at_s;
    s_left = static_cast<uint64_t>(A.units) * s_step - at_s;
    slabs = 2 * (ue - ub);
  }
  // To the next slab; behind the tile's last one it stays there.
  template <bool ODD>
  __device__ __forceinline__ void advance() {
    --slabs;
    const bool on = slabs > 0;
    const uint32_t da = on ? a_step : 0u, db = on ? b_step : 0u;
    a += da;
    a_left -= da;
    b += db;
    b_left -= db;
    if constexpr (ODD) {
      const uint32_t ds = on ? s_step : 0u;
      s += ds;
      s_left -= ds;
    }
  }
};

// This lane's byte offsets in a wave's loads.
struct Offsets {
  int a, b, s;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(uint64_t at, uint64_t left) {
  return make_rsrc(reinterpret_cast<const void*>(at), 0, clip(left));
}

// The loads that bring this wave's share of a slab into a stage: the codes of A and
// of B, 16 rows each.
template <class T>
__device__ __forceinline__ void load_slab(typename T::Stage& st, const Stream& S, const Offsets& off, int wave) {
  constexpr int RA = T::TM / 4, RB = T::TN / 4;  // rows of this wave
  const __amdgpu_buffer_rsrc_t ca = resource(S.a, S.a_left), cb = resource(S.b, S.b_left);
  lds_ptr_t da = (lds_ptr_t)(st.code + wave * RA * 4), db = (lds_ptr_t)(st.code + (T::TM + wave * RB) * 4);
#define FP8_LOAD(R, RSRC, DST, VOFF, PIECE)     \
  if constexpr ((PIECE) * 1024 < (R) * 64)      \
    __builtin_amdgcn_raw_ptr_buffer_load_lds(RSRC, DST, 16, VOFF, 0, (PIECE) * 1024, 0)
  FP8_LOAD(RA, ca, da, off.a, 0);
  FP8_LOAD(RA, ca, da, off.a, 1);
  FP8_LOAD(RA, ca, da, off.a, 2);
  FP8_LOAD(RA, ca, da, off.a, 3);
  FP8_LOAD(RB, cb, db, off.b, 0);
  FP8_LOAD(RB, cb, db, off.b, 1);
  FP8_LOAD(RB, cb, db, off.b, 2);
  FP8_LOAD(RB, cb, db, off.b, 3);
#undef FP8_LOAD
  static_assert(RA % 16 == 0 && RB % 16 == 0 && RA <= 64 && RB <= 64, "loads of a slab");
}

// One load: even waves bring A's scales of the unit that the slab begins, odd ones B's,
// two of them the same bytes, so that every wave has the same loads under way.
// Lanes behind the tile's rows have an offset behind the matrix and write zeros.
__device__ __forceinline__ void load_scales(ScaleStage& st, const Stream& S, const Offsets& off, int wave) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(resource(S.s, S.s_left), (lds_ptr_t)((wave & 1) != 0 ? st.b : st.a), 16, off.s, 0,
                                           0, 0);
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
// of the next slab (stage `nxt`) there.  The slab 4 ahead is loaded into `cur` and,
// in even slabs, its unit's scales into `sc`; odd slabs read the next unit's scales
// from `sc`.  Loads and reads are spread over the MFMAs (a burst of them would hold
// up the wave, which issues in order).  kStores: stores that were issued behind the
// loads that are waited for.
template <class T, int FA, bool EXACT, bool ODD, int kStores>
__device__ __forceinline__ void slab(f32x16_t (&acc)[T::FN][T::FM], Frags<T>& f, Scales<T>& w, Wide<T>& v,
                                     typename T::Stage& cur, const typename T::Stage& nxt, ScaleStage& sc, Stream& S,
                                     const Offsets& off, int wave, int lane, const Reads& at) {
  constexpr int M = T::FM * T::FN, kLoads = T::kCodeLoads + (ODD ? 0 : 1);
  constexpr int kReads = (ODD ? 3 : 2) * (T::FM + T::FN);
  constexpr int kAhead = 2 * T::kCodeLoads + 1;  // loads of two slabs
  // this wave's part of the next slab has landed (two slabs stay under way), and all
  // its reads of this one are done
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(kAhead + kStores < 63 ? kAhead + kStores : 63, 0));
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  Frags<T> fn;
  Scales<T> wn;
  load_slab<T>(cur, S, off, wave);
  if constexpr (!ODD) load_scales(sc, S, off, wave);
  read_frag<T::FN>(fn.b, nxt, at.b, lane);
  read_frag<T::FM>(fn.a, nxt, at.a, lane);
  if constexpr (ODD) {
    read_scales<T::FN>(wn.b, sc.b, at.sb, lane);
    read_scales<T::FM>(wn.a, sc.a, at.sa, lane);
  }
  S.template advance<ODD>();
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

// The LDS of a block.  (The stages are objects of their own so that the compiler can
// tell a read of one from a load into another.)
template <class T>
struct Lds {
  typename T::Stage &s0, &s1, &s2, &s3;
  ScaleStage &c0, &c1;
  uint4* out;  // where a block stays: 32 rows of 128 bytes for each wave's results
};
constexpr int kOutPitch = 9;  // uint4 of such a row, one against bank conflicts
#define FP8_LDS(T)                                                              \
  __shared__ typename T::Stage s0, s1, s2, s3;                                  \
  __shared__ ScaleStage c0, c1;                                                 \
  __shared__ uint4 out_stage[T::kStays ? 4 * 32 * kOutPitch : 1];               \
  const Lds<T> lds{s0, s1, s2, s3, c0, c1, out_stage}

// A tile of a launch: rows of A and of B, and units ub .. ue - 1 (one at least).
struct Work {
  Operand A, B;
  int ub, ue;
  void* C;
  int rows, cols;    // the ends of its rows and columns in C, whose rows are `cols` long
  int add;           // C is added to
  int sums;          // C holds fp32 sums of a piece of k
};

// A wave's accumulators to C; fp32 C for exact sums.
template <class T, bool EXACT, bool ADD>
__device__ __forceinline__ void store_product(const Work& t, const f32x16_t (&acc)[T::FN][T::FM], uint4* stage, int i, int j,
                                              int lane) {
  constexpr int DC = EXACT ? kF32 : kBF16;
  static_assert(EXACT || !T::kStays, "blocks that stay are for fp32 results");
  constexpr int XS = T::kStays ? 1 : T::FN;  // rows of 128 bytes, where a block stays
  store_tile<T, DC, ADD, XS>(t.C, acc, stage, i, j, t.rows, t.cols, lane);
}

// All the block's tiles: find(&id, &work) is the first tile of the launch from the id-th
// on, in steps of gridDim.x, if there is one.
template <class T, int FA, bool EXACT, class Find>
__device__ __forceinline__ void take_tiles(const Lds<T>& lds, const Find& find, int wave, int lane) {
  // lane l fills slot l % 4 of row l / 4 of each 16-row run
  const int vcode = (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 4) & 3)) * 16);
  const int lines = ((wave & 1) != 0 ? T::TN : T::TM) / kF8Line + 1;
  const Offsets off{wave * (T::TM / 4) * 64 + vcode, wave * (T::TN / 4) * 64 + vcode, lane < lines ? lane * 16 : 0x7ffffff0};
  const int ra = T::FM * 32 * (wave / T::WN), rb = T::FN * 32 * (wave % T::WN);

  int id = blockIdx.x;
  Work t;
  if (!find(&id, &t)) return;
  Stream S;  // always a round of the ring ahead of the products
  S.start(t.A, t.B, t.ub, t.ue, wave);
  load_slab<T>(lds.s0, S, off, wave);
  load_scales(lds.c0, S, off, wave);
  S.template advance<false>();
  load_slab<T>(lds.s1, S, off, wave);
  S.template advance<true>();
  load_slab<T>(lds.s2, S, off, wave);
  load_scales(lds.c1, S, off, wave);
  S.template advance<false>();
  load_slab<T>(lds.s3, S, off, wave);
  S.template advance<true>();
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(3 * T::kCodeLoads + 1, 0));  // the first slab has landed
  asm volatile("s_barrier" ::: "memory");
  // One slab of a wave that has no rows or columns of the tile: only its loads.
  const auto pass = [&](auto odd, typename T::Stage& stage, ScaleStage& sc) {
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(2 * T::kCodeLoads + 1, 0));
    asm volatile("s_barrier" ::: "memory");
    load_slab<T>(stage, S, off, wave);
    if constexpr (!decltype(odd)::value) load_scales(sc, S, off, wave);
    S.template advance<decltype(odd)::value>();
  };
  constexpr std::false_type kEvenSlab;
  constexpr std::true_type kOddSlab;
  bool full = false;  // the last tile had all its stores
  for (;;) {
    const int i = t.A.row + ra, j = t.B.row + rb;  // this wave's first row and column
    // what the last round loads: the next tile's first one, or anything
    Work n = t;
    bool more = false;
    if constexpr (T::kStays) {
      id += gridDim.x;
      more = find(&id, &n);
      if (!more) n = t;  // whatever the search left there may lie behind the matrices
    }
    Stream N;
    N.start(n.A, n.B, n.ub, n.ue, wave);
    int units = t.ue - t.ub;
    // groups end anywhere in a tile: half of the last tiles' waves have nothing to do,
    // and leave their power to the others
    if (i >= t.rows || j >= t.cols) {
      for (; units > 0; units -= 2) {
        if (units <= 2) S = N;
        pass(kEvenSlab, lds.s0, lds.c0);
        pass(kOddSlab, lds.s1, lds.c1);
        if (T::kStays || units >= 2) {
          pass(kEvenSlab, lds.s2, lds.c1);
          pass(kOddSlab, lds.s3, lds.c0);
        }
      }
      if constexpr (!T::kStays) {
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
        asm volatile("s_barrier" ::: "memory");  // the others' in front of their results
      }
      if (!more) break;
      full = false;
      t = n;
      continue;
    }
    f32x16_t acc[T::FN][T::FM] = {};
    // the first slab is in s0: the last barrier stood behind its loads
    const Reads at{ra, T::TM + rb, (t.A.row & (kF8Line - 1)) + ra, (t.B.row & (kF8Line - 1)) + rb};
    Frags<T> f;
    Scales<T> w;
    Wide<T> v;
    __builtin_amdgcn_sched_barrier(0);
    read_frag<T::FN>(f.b, lds.s0, at.b, lane);
    read_frag<T::FM>(f.a, lds.s0, at.a, lane);
    read_scales<T::FN>(w.b, lds.c0.b, at.sb, lane);
    read_scales<T::FM>(w.a, lds.c0.a, at.sa, lane);
    if constexpr (EXACT) widen<T, FA, 0>(v, f, w);
    const auto round = [&](auto stores) {
      constexpr int kStores = decltype(stores)::value;
      if (units == 2) S = N;
      slab<T, FA, EXACT, false, kStores>(acc, f, w, v, lds.s0, lds.s1, lds.c0, S, off, wave, lane, at);
      slab<T, FA, EXACT, true, kStores>(acc, f, w, v, lds.s1, lds.s2, lds.c1, S, off, wave, lane, at);
      slab<T, FA, EXACT, false, kStores>(acc, f, w, v, lds.s2, lds.s3, lds.c1, S, off, wave, lane, at);
      slab<T, FA, EXACT, true, 0>(acc, f, w, v, lds.s3, lds.s0, lds.c0, S, off, wave, lane, at);
      units -= 2;
    };
    // the loads that the first round waits for were issued before the stores of the
    // tile before; if it had all of them, they need not have ended
    if constexpr (T::kStays)
      if (full && units >= 2) round(std::integral_constant<int, T::kStores>());
    while (units >= 2) round(std::integral_constant<int, 0>());
    if (units > 0) {
      S = N;
      slab<T, FA, EXACT, false, 0>(acc, f, w, v, lds.s0, lds.s1, lds.c0, S, off, wave, lane, at);
      slab<T, FA, EXACT, true, 0>(acc, f, w, v, lds.s1, lds.s2, lds.c1, S, off, wave, lane, at);
      if constexpr (T::kStays) {
        // the two slabs that were loaded for nothing give way to others
        pass(kEvenSlab, lds.s2, lds.c1);
        pass(kOddSlab, lds.s3, lds.c0);
      }
    }
    uint4* stage = lds.out + wave * 32 * kOutPitch;
    if constexpr (!T::kStays) {
      // loads behind the last unit are still on their way into LDS: they end here,
      // and so do all waves' reads, before LDS takes the results
      __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
      asm volatile("s_barrier" ::: "memory");
      stage = (wave == 0 ? lds.s0 : wave == 1 ? lds.s1 : wave == 2 ? lds.s2 : lds.s3).code;
      if (t.sums) {
        store_tile<T, kF32, false>(t.C, acc, stage, i, j, t.rows, t.cols, lane);
        return;
      }
    }
    if (t.add) {
      store_product<T, EXACT, true>(t, acc, stage, i, j, lane);
    } else {
      store_product<T, EXACT, false>(t, acc, stage, i, j, lane);
    }
    if (!more) break;
    full = i + 32 * T::FM <= t.rows && j + 32 * T::FN <= t.cols;
    t = n;
  }
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));  // loads into this block's LDS end with it
}

// `bytes` bytes from p on (both even) to zero, shared by the launch's blocks.
__device__ __forceinline__ void clear_bytes(void* p, int64_t bytes) {
  const uintptr_t begin = reinterpret_cast<uintptr_t>(p), end = begin + bytes;
  uintptr_t head = (begin + 15) & ~uintptr_t{15}, tail = end & ~uintptr_t{15};
  if (head > tail) head = tail = end;
  const int64_t me = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, all = static_cast<int64_t>(gridDim.x) * 256;
  for (uintptr_t q = head + me * 16; q < tail; q += all * 16) *reinterpret_cast<uint4*>(q) = make_uint4(0, 0, 0, 0);
  if (me < 16) {  // at most 7 elements of two bytes at either end (15 without a middle)
    if (begin + me * 2 < head) *reinterpret_cast<uint16_t*>(begin + me * 2) = 0;
    if (tail + me * 2 < end) *reinterpret_cast<uint16_t*>(tail + me * 2) = 0;
  }
}

typedef Tile<256, 256, 2> Big;
typedef Tile<256, 256, 2, true> Staying;
typedef Tile<128, 128, 2> Mid;
typedef Tile<64, 128, 1> Low;

template <class T>
constexpr int kBlocksPerCU = T::TM == 256 ? 1 : 2;
template <class T>
uint32_t blocks_of(int64_t tiles) {
  return static_cast<uint32_t>(T::kStays && tiles > kCUs ? kCUs : tiles);
}

// Whether 256 x 256 tiles take less time than 128 x 128 ones, by what was measured of
// both (us, bf16 results; fp32 ones take 1.85 times both).  A 256 x 256 tile takes 1.42 a
// unit and 10 that nothing of its compute unit overlaps (the first loads, the
// results), by whole rounds of 256 tiles; where compute units are left without work
// the others have their power, so that half of what is missing counts.  128 x 128
// tiles, two blocks a compute unit and rounds of a quarter, take 1.77 and 6 for the
// same area.  work: elements of C in 256 x 256; big, mid: tiles of either size.
inline bool big_tiles_pay(double work, double big, double mid, int units, double mid_slower) {
  const double rounds = std::ceil(big / kCUs);
  const double big_us = (work / kCUs + rounds) / 2 * 1.42 * units + 10.0 * rounds;
  return big_us <= (work + mid / 4) / 2 / kCUs * (1.77 * units + 6.0) * mid_slower;
}

}  // namespace fp8
}  // namespace muon

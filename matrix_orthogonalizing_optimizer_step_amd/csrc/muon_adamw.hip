// The AdamW step over a list of tensors of any sizes, for the parameters that
// are not hidden 2-D weights (embeddings, head, norms, biases), with the two
// moments in fp32 or in 8-bit codes, and the host side of its entry points.
//
//   g = s G,  m <- b1 m + (1 - b1) g,  v <- b2 v + (1 - b2) g^2,
//   W <- W - lr ((m / (1 - b1^t)) / (sqrt(v) / sqrt(1 - b2^t) + eps) + wd W)
//
// (AdamW update [MuonBlog §1], weight decay decoupled as in the Muon update.)
// All arithmetic is fp32; a bf16 W is rounded once, to nearest even.
//
// One launch covers a list of up to 87 (64) tensors: each is cut into chunks, one
// block per chunk, and a block finds its tensor in the chunk starts that travel
// with the kernel arguments, as the pointers do (no table in memory, so nothing
// has to be copied to the device first and a captured graph holds everything).
//
// With 32-bit states memory bounds the step: an element is read and written once,
// 28 bytes with fp32 W and G, against some 25 instructions.  What counts is bytes
// in flight: a thread issues all loads of its 16 elements before it uses one, and
// the chip holds thousands of such blocks.  With 8-bit states it is 10.1 bytes
// (bf16 W and G) against 58 vector instructions, 3 of them at a quarter of the rate,
// and both count: 235M parameters with 71 instructions 439 us, with 58 428, then with
// accesses past the caches 384.
//
// Accesses go past the caches: a training step lies between two calls, so nothing
// of the call before is left there.  With cold caches that is as fast or faster at
// almost every size, in us past / through them: 32-bit states, fp32 W and G 1M
// elements 10.2 / 12.0, 12M 62.5 / 66.8, 24M 121 / 121, 96M 479 / 503 (24M with bf16
// G 114 / 110); 8-bit states, bf16 W and G 1M 8.9 / 9.4, 24M 48.0 / 51.5, 96M 168 /
// 180.  Called again and again on 0.55 GB, which then stay in the 256 MB cache in
// part, the 32-bit step would be 12 % faster through them.
//
// Measured on 235M parameters: 32-bit states 5.83 TB/s (bf16 W and
// G, 886 us) and 5.90 (fp32, 1114 us), 8-bit states 6.2 (384 us) and 5.70 (665 us);
// a large copy reaches 4.8 and an addition in place 6.0.
#include <math.h>
#include <string.h>

#include <type_traits>

#include "../../include/muon.h"
#include "muon_convert.h"
#include "muon_internal.h"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kQuads = 4;                              // 4-element pieces per thread, 32-bit states
constexpr int kChunk32 = kThreads * 4 * kQuads;        // elements per block, 32-bit states
constexpr int kGroup = 128;                            // elements per scale, 8-bit states
constexpr int kChunk8 = kThreads * 8;                  // elements per block, 8-bit states (16 groups)

struct AdamwScalars {
  float lr, wd, eps, b1, ob1, b2, ob2;
  float c1, c2;              // 1 / (1 - b1^t), 1 / sqrt(1 - b2^t) for the host's t
  float lr1, wd1;            // lr c1, wd / c1
  double beta1, beta2;
  int64_t step;
  const int64_t* step_dev;   // t in device memory, or null
  const float* grad_scale;   // s in device memory, or null (1)
  uint32_t seed;
  int small_eps;             // 8-bit states: eps lets errors of the smallest roots be seen
};

// The tensors of one launch, up to K of them with P pointers each.  Two sizes of
// the kernel arguments: as many tensors as keep them within the 4 KB that a
// launch takes, and kFew for short lists, whose 0.5 KB the host copies sooner
// (a call on one norm 4.87 -> 4.65 us).
constexpr int kFew = 8;
constexpr int many_tensors(int pointers) { return 3840 / (8 * pointers + 12); }

template <int P, int K>
struct Lists {
  int count;              // tensors in this launch
  int first;              // list index of the first one
  uint32_t start[K + 1];  // first block of each tensor
  int64_t size[K];
  void* ptr[P][K];
};

constexpr int kPtrs32 = 4;  // W, G, M, V
constexpr int kPtrs8 = 6;   // W, G, codes and scales of m, codes and scales of the root of v

template <int P, int K>
struct AdamwArgs {
  AdamwScalars s;
  Lists<P, K> t;
};
static_assert(sizeof(AdamwArgs<kPtrs32, many_tensors(kPtrs32)>) <= 4096 &&
              sizeof(AdamwArgs<kPtrs8, many_tensors(kPtrs8)>) <= 4096, "kernel arguments");

// The tensor of this block (the last one whose start is not beyond it; empty
// tensors have the next one's start and are passed over).
template <int P, int K>
__device__ __forceinline__ int find_tensor(const Lists<P, K>& t, uint32_t block) {
  int lo = 0, hi = t.count;  // start[lo] <= block < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.start[mid] <= block) {
      lo = mid;
    } else {
      hi = mid;
    }
  }
  return lo;
}

__device__ __forceinline__ double int_power(double b, int64_t t) {
  double r = 1.0;
  for (; t > 0; t >>= 1) {
    if (t & 1) r *= b;
    b *= b;
  }
  return r;
}

// The scalars with a step number or a gradient scale from device memory.  With t from
// there every thread takes the powers itself, before its loads: 8-bit states and bf16
// // 235M parameters 380 -> 425 us, 25M 43.5 -> 49, a small call 4.7 -> 5.3.  With fp32 W
// (661 / 657) or 32-bit states (bf16 884 / 886) memory hides it.
struct Scalars {
  float c1, c2, lr1, wd1, gs;
  int64_t step;
};
__device__ __forceinline__ Scalars load_scalars(const AdamwScalars& s) {
  Scalars r{s.c1, s.c2, s.lr1, s.wd1, 1.0f, s.step};
  if (s.step_dev != nullptr) {
    const int64_t t = *s.step_dev;
    r.step = t < 1 ? 1 : t;
    const double left = 1.0 - int_power(s.beta1, r.step);
    r.c1 = static_cast<float>(1.0 / left);
    r.lr1 = static_cast<float>(s.lr / left);
    r.wd1 = static_cast<float>(s.wd * left);
    r.c2 = static_cast<float>(1.0 / sqrt(1.0 - int_power(s.beta2, r.step)));
  }
  if (s.grad_scale != nullptr) r.gs = *s.grad_scale;
  return r;
}

// N consecutive elements of dtype D (N a multiple of 4) as loaded, so that a
// thread has all its loads out before it waits for the first.  Tensors may start
// anywhere (views into flat buffers): the loads and stores are 16 bytes wide
// (8 for four 16-bit elements) but need the alignment of one element only.
// `left` elements are there (all N if FULL); the others read as zero and are not
// written.
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef u32x2_t u32x2_a1 __attribute__((aligned(1)));
typedef u32x2_t u32x2_a2 __attribute__((aligned(2)));
typedef u32x4_t u32x4_a2 __attribute__((aligned(2)));
typedef u32x4_t u32x4_a4 __attribute__((aligned(4)));

template <int D, int N>
struct Raw {
  uint32_t v[D == kF32 ? N : N / 2];
};

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

template <int D, int N, bool FULL, bool NT = false>
__device__ __forceinline__ Raw<D, N> load_raw(const void* p, int64_t i, int64_t left) {
  Raw<D, N> r;
  if (FULL || left >= N) {
    if constexpr (D == kF32) {
#pragma unroll
      for (int q = 0; q < N; q += 4) {
        const u32x4_t x = LOAD_VEC(reinterpret_cast<const u32x4_a4*>(static_cast<const float*>(p) + i + q));
#pragma unroll
        for (int k = 0; k < 4; ++k) r.v[q + k] = x[k];
      }
    } else if constexpr (N == 4) {
      const u32x2_t x = LOAD_VEC(reinterpret_cast<const u32x2_a2*>(static_cast<const uint16_t*>(p) + i));
      r.v[0] = x[0];
      r.v[1] = x[1];
    } else {
#pragma unroll
      for (int q = 0; q < N; q += 8) {
        const u32x4_t x = LOAD_VEC(reinterpret_cast<const u32x4_a2*>(static_cast<const uint16_t*>(p) + i + q));
#pragma unroll
        for (int k = 0; k < 4; ++k) r.v[q / 2 + k] = x[k];
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < (D == kF32 ? N : N / 2); ++k) r.v[k] = 0;
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (k < left) {
        if constexpr (D == kF32) {
          r.v[k] = static_cast<const uint32_t*>(p)[i + k];
        } else {
          r.v[k >> 1] |= static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i + k]) << (16 * (k & 1));
        }
      }
  }
  return r;
}

template <int D, int N>
__device__ __forceinline__ float raw_value(const Raw<D, N>& r, int k) {
  if constexpr (D == kF32) {
    return __uint_as_float(r.v[k]);
  } else {
    const uint16_t h = static_cast<uint16_t>((k & 1) ? r.v[k >> 1] >> 16 : r.v[k >> 1]);
    return D == kBF16 ? bf16_to_f32(h) : f16_to_f32(h);
  }
}

template <int D, int N, bool FULL, bool NT = false>
__device__ __forceinline__ void store_values(void* p, int64_t i, int64_t left, const float (&x)[N]) {
  if (FULL || left >= N) {
    if constexpr (D == kF32) {
#pragma unroll
      for (int q = 0; q < N; q += 4)
        STORE_VEC(reinterpret_cast<u32x4_a4*>(static_cast<float*>(p) + i + q),
                  __builtin_bit_cast(u32x4_t, make_float4(x[q], x[q + 1], x[q + 2], x[q + 3])));
    } else if constexpr (N == 4) {
      STORE_VEC(reinterpret_cast<u32x2_a2*>(static_cast<uint16_t*>(p) + i),
                ((u32x2_t){f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3])}));
    } else {
#pragma unroll
      for (int q = 0; q < N; q += 8)
        STORE_VEC(reinterpret_cast<u32x4_a2*>(static_cast<uint16_t*>(p) + i + q),
                  ((u32x4_t){f32x2_to_bf16x2(x[q], x[q + 1]), f32x2_to_bf16x2(x[q + 2], x[q + 3]),
                             f32x2_to_bf16x2(x[q + 4], x[q + 5]), f32x2_to_bf16x2(x[q + 6], x[q + 7])}));
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (k < left) store_from_f32(p, i + k, D, x[k]);
  }
}

// One element's moments and weight.  The moments' products and sums are
// rounded one at a time: their codes (8-bit states) then do not depend on what a
// compiler fuses.
__device__ __forceinline__ void update(float& w, float g, float& m, float& v, const AdamwScalars& s, const Scalars& r) {
#pragma clang fp contract(off)
  g *= r.gs;
  m = s.b1 * m + s.ob1 * g;
  v = s.b2 * v + (s.ob2 * g) * g;
  w = w - s.lr * (m * r.c1 / (sqrtf(v) * r.c2 + s.eps) + s.wd * w);
}

template <int DW, int DG, bool FULL>
__device__ __forceinline__ void adamw_chunk(void* W, const void* G, void* M, void* V, int64_t base, int64_t n,
                                            const AdamwScalars& s, const Scalars& r) {
  Raw<DW, 4> w4[kQuads];
  Raw<DG, 4> g4[kQuads];
  Raw<kF32, 4> m4[kQuads], v4[kQuads];
#pragma unroll
  for (int q = 0; q < kQuads; ++q) {
    const int64_t i = base + (q * kThreads + static_cast<int>(threadIdx.x)) * 4;
    w4[q] = load_raw<DW, 4, FULL, true>(W, i, n - i);
    g4[q] = load_raw<DG, 4, FULL, true>(G, i, n - i);
    m4[q] = load_raw<kF32, 4, FULL, true>(M, i, n - i);
    v4[q] = load_raw<kF32, 4, FULL, true>(V, i, n - i);
  }
#pragma unroll
  for (int q = 0; q < kQuads; ++q) {
    const int64_t i = base + (q * kThreads + static_cast<int>(threadIdx.x)) * 4;
    float w[4], m[4], v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      w[k] = raw_value(w4[q], k);
      m[k] = raw_value(m4[q], k);
      v[k] = raw_value(v4[q], k);
      update(w[k], raw_value(g4[q], k), m[k], v[k], s, r);
    }
    store_values<kF32, 4, FULL, true>(M, i, n - i, m);
    store_values<kF32, 4, FULL, true>(V, i, n - i, v);
    store_values<DW, 4, FULL, true>(W, i, n - i, w);
  }
}

template <int DW, int DG, int K>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamwArgs<kPtrs32, K> a) {
  const int t = find_tensor(a.t, blockIdx.x);
  const int64_t n = a.t.size[t], base = static_cast<int64_t>(blockIdx.x - a.t.start[t]) * kChunk32;
  const Scalars r = load_scalars(a.s);
  if (base + kChunk32 <= n) {
    adamw_chunk<DW, DG, true>(a.t.ptr[0][t], a.t.ptr[1][t], a.t.ptr[2][t], a.t.ptr[3][t], base, n, a.s, r);
  } else {
    adamw_chunk<DW, DG, false>(a.t.ptr[0][t], a.t.ptr[1][t], a.t.ptr[2][t], a.t.ptr[3][t], base, n, a.s, r);
  }
}

// ---------------------------------------------------------------------------
// 8-bit states: per group of 128 consecutive elements of a tensor (the last
// group of a tensor may be shorter) m = c_m s_m and sqrt(v) = c_r s_r with
// codes c in e4m3 and fp32 scales s = (largest magnitude of the group) / 448.
// e4m3 keeps a relative precision of 2^-4 over 2^14.8 below the largest value,
// and 2^-9 absolute under it; the root of v is kept, not v, because the update
// divides by the root and the same code then spans the square of that range.
//
// c_m is rounded to nearest: with b1 = 0.9 a step moves m by a tenth, more
// than half a code step (1/16).  c_r cannot be: a step moves v by 1 - b2 =
// 1e-3 of itself, so to nearest it would stand still from about the tenth step
// on.  It goes to one of its two neighbours lo <= x < hi with the chance that
// keeps the expected square: up when (x - lo)(x + lo) > u (hi - lo)(hi + lo)
// (rounding at random in the root itself would raise v by the variance at
// every step).  u comes from a hash of (seed, t, tensor, element), so a step
// is reproducible.  A positive v never gets code 0: the update would then
// divide by eps alone.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  // xor-shift and multiply rounds; the constants are odd numbers near 2^32 times
  // the golden ratio's inverse and 2^32 times (e - 2)
  x ^= x >> 16;
  x *= 0x9E3779B1u;
  x ^= x >> 15;
  x *= 0xB7E15163u;
  return x ^ (x >> 16);
}

// The two halves of mix(x) as 2^32 u = 65536 (half + 1/2), lower half first.
__device__ __forceinline__ void mix_chances(uint32_t x, float* lo, float* hi) {
  x ^= x >> 16;
  x *= 0x9E3779B1u;
  x ^= x >> 15;
  x *= 0xB7E15163u;
  *lo = static_cast<float>((x << 16 | 0x8000u) ^ (x & 0xFFFF0000u));
  *hi = static_cast<float>((x & 0xFFFF0000u) | 0x8000u);
}

// 1 / s rounded to nearest, or 0 where the group is stored as zeros (s zero or
// not finite).  v_rcp_f32 is off by one unit at most and one Newton step ends
// the error.
__device__ __forceinline__ float code_inverse(float s) {
  const float r = __builtin_amdgcn_rcpf(s);
  return s > 0.0f && s < INFINITY ? fmaf(fmaf(-s, r, 1.0f), r, r) : 0.0f;
}

// The scale of a group from its largest magnitude.  A scale under 2^-126 is
// taken as 0.
__device__ __forceinline__ float code_scale(float top) {
  const float s = top * (1.0f / 448.0f);
  return s < 0x1p-126f ? 0.0f : s;
}

// sqrt(x) rounded to nearest, for x zero or finite and at least 2^-102: s = x /
// sqrt(x) by v_rsq_f32 and one Newton step with the residual x - s^2, which fmaf gives
// exactly.  From 2^-126 to 2^-102 the residual is rounded to 2^-149, which adds 2^-25
// of the root at most.  Subnormal x: between 0 and the root, which is under 2^-63, and
// off by at most 2^-64.  Infinity and NaN: NaN.
__device__ __forceinline__ float root_nearest(float x) {
  const uint32_t bits = __float_as_uint(x);
  const float r = __builtin_amdgcn_rsqf(__uint_as_float(bits > 0x00800000u ? bits : 0x00800000u));
  const float s = x * r;
  return fmaf(fmaf(-s, s, x), 0.5f * r, s);
}

// The value of the code of x in [0, 448 (1 + 2^-22)] (see above), given 2^32 u.
// In units of the code step at x (a power of two, so nothing is
// rounded by it) the neighbours are f and f + 1, and the condition is (y - f)
// (y + f) > u (2 f + 1).  Of 14 units of 32, the largest code, 14 (1 + 2^-22) is
// 14 for every u: (y - f)(y + f) < 2^-13 < 29 * 2^-17.
__device__ __forceinline__ float root_code_value(float x, float u32, bool positive) {
  const uint32_t binade = __float_as_uint(x) & 0x7F800000u;
  const uint32_t b = binade > (121u << 23) ? binade : 121u << 23;  // of x, at least 2^-6; the step is 1/8 of it
  const float y = x * __uint_as_float((257u << 23) - b);           // x / step: 8..16, or 0..8 under 2^-6
  const float f = floorf(y);
  const float bar = u32 * fmaf(f, 0x1p-31f, 0x1p-32f);
  const bool up = ((y - f) * (y + f) > bar) | ((f == 0.0f) & positive);
  const float step = __uint_as_float(b - (3u << 23));
  return fmaf(f, step, up ? step : 0.0f);
}

// One element's moments as in update(); its weight, with the root of the new v,
// by W - (lr c1) (m / (root c2 + eps) + (wd / c1) W), the quotient by v_rcp_f32
// (off by one unit at most).
__device__ __forceinline__ void moments8(float g, float& m, float& v, const AdamwScalars& s) {
#pragma clang fp contract(off)
  m = s.b1 * m + s.ob1 * g;
  v = s.b2 * v + (s.ob2 * g) * g;
}
__device__ __forceinline__ float weight8(float w, float m, float root, const AdamwScalars& s, const Scalars& r) {
  const float inverse = __builtin_amdgcn_rcpf(fmaf(root, r.c2, s.eps));
  return fmaf(-r.lr1, fmaf(r.wd1, w, m * inverse), w);
}

// Largest magnitude of 16 threads' 8 values each (a DPP row), compared as unsigned
// integers across the threads: a NaN's bits count as the largest.
__device__ __forceinline__ float group_max(const float (&v)[8]) {
  float top = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; k += 2)
    top = __builtin_elementwise_maximum(__builtin_elementwise_maximum(fabsf(v[k]), fabsf(v[k + 1])), top);
  uint32_t x = __float_as_uint(top);
  const auto rotate_max = [&](auto turn) {
    const uint32_t y = static_cast<uint32_t>(
        __builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x120 + decltype(turn)::value, 0xf, 0xf, true));
    x = x > y ? x : y;
  };
  rotate_max(std::integral_constant<int, 1>());
  rotate_max(std::integral_constant<int, 2>());
  rotate_max(std::integral_constant<int, 4>());
  rotate_max(std::integral_constant<int, 8>());
  return __uint_as_float(x);
}

// 8 code bytes.
template <bool FULL>
__device__ __forceinline__ u32x2_t load_codes(const void* p, int64_t i, int64_t left) {
  const uint8_t* c = static_cast<const uint8_t*>(p) + i;
  if (FULL || left >= 8) return __builtin_nontemporal_load(reinterpret_cast<const u32x2_a1*>(c));
  u32x2_t r = {0, 0};
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < left) r[k >> 2] |= static_cast<uint32_t>(c[k]) << (8 * (k & 3));
  return r;
}
template <bool FULL>
__device__ __forceinline__ void store_codes(void* p, int64_t i, int64_t left, u32x2_t x) {
  uint8_t* c = static_cast<uint8_t*>(p) + i;
  if (FULL || left >= 8) {
    __builtin_nontemporal_store(x, reinterpret_cast<u32x2_a1*>(c));
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < left) c[k] = static_cast<uint8_t>(x[k >> 2] >> (8 * (k & 3)));
  }
}

// One chunk, from element `base` on: 8 elements a thread, 16 threads a group.  Of
// fp32 a thread has two halves of 16 bytes, so that two loads share each cache line,
// and W and G in fp32 go through the caches (235M elements 664 us, past them 692).
template <int DW, int DG, bool FULL, int K>
__device__ __forceinline__ void adamw8_chunk(const AdamwArgs<kPtrs8, K>& a, int t, int64_t base, int64_t n, const Scalars& r) {
  // the block's pointers are scalars and a thread's offset has 32 bits
  const int i = 8 * static_cast<int>(threadIdx.x), group = static_cast<int>(threadIdx.x) >> 4;
  char* const W = static_cast<char*>(a.t.ptr[0][t]) + base * (DW == kF32 ? 4 : 2);
  const char* const G = static_cast<const char*>(a.t.ptr[1][t]) + base * (DG == kF32 ? 4 : 2);
  char* const mc = static_cast<char*>(a.t.ptr[2][t]) + base;
  char* const rc = static_cast<char*>(a.t.ptr[4][t]) + base;
  float* const ms = static_cast<float*>(a.t.ptr[3][t]) + base / kGroup;
  float* const rs = static_cast<float*>(a.t.ptr[5][t]) + base / kGroup;
  const int64_t left = n - base - i;  // 0 or less: nothing is there, but the group's other threads may need this one
  const Raw<DW, 8> w8 = load_raw<DW, 8, FULL, DW != kF32>(W, i, left);
  const Raw<DG, 8> g8 = load_raw<DG, 8, FULL, DG != kF32>(G, i, left);
  const u32x2_t cm = load_codes<FULL>(mc, i, left), cr = load_codes<FULL>(rc, i, left);
  const bool any = FULL || left > 0;
  const float sm = any ? ms[group] : 0.0f, sr = any ? rs[group] : 0.0f;
  float g[8], m[8], v[8], root[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) g[k] = raw_value(g8, k);
  if (a.s.grad_scale != nullptr) {
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] *= r.gs;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t cmk = cm[k >> 2], crk = cr[k >> 2];
    const auto pm = (k & 2) ? __builtin_amdgcn_cvt_pk_f32_fp8(cmk, true) : __builtin_amdgcn_cvt_pk_f32_fp8(cmk, false);
    const auto pr = (k & 2) ? __builtin_amdgcn_cvt_pk_f32_fp8(crk, true) : __builtin_amdgcn_cvt_pk_f32_fp8(crk, false);
    m[k] = pm[k & 1] * sm;
    const float old = pr[k & 1] * sr;
    v[k] = old * old;
    moments8(g[k], m[k], v[k], a.s);
    root[k] = root_nearest(v[k]);
  }
  // the places of a tensor's last group behind its end hold zeros (codes and
  // gradients), which stay zeros and leave the group's largest values alone
  const float group_m = group_max(m);
  float group_root = group_max(root);
  // In a group whose largest root is 2^-33 or more, one under 2^-51 (1 + 2^-23) gets
  // the smallest code whatever it is exactly: 448 * 2^-18 is under the code step
  // 2^-9.  Smaller roots, infinities and NaN take the general function.  The weight is
  // divided by the root itself: where eps does not hide what the short root is off by
  // (see small_eps in make_scalars), small roots are taken again (235M bf16
  // parameters: without such roots no slower, with nothing but such roots beside one
  // large one in each group 401 us for 384).
  if (!((group_root >= 0x1p-33f && group_root < INFINITY) || group_root == 0.0f)) {
#pragma unroll
    for (int k = 0; k < 8; ++k) root[k] = sqrtf(v[k]);
    group_root = group_max(root);
  } else if (a.s.small_eps) {
    bool small = false;
#pragma unroll
    for (int k = 0; k < 8; ++k) small |= v[k] > 0.0f && v[k] < 0x1p-102f;
    if (small) {
#pragma unroll
      for (int k = 0; k < 8; ++k) root[k] = sqrtf(v[k]);
    }
  }
  float w[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k] = weight8(raw_value(w8, k), m[k], root[k], a.s, r);
  store_values<DW, 8, FULL, DW != kF32>(W, i, left, w);
  const float sm2 = code_scale(group_m), sr2 = code_scale(group_root);
  const float im = code_inverse(sm2), ir = code_inverse(sr2);
  const uint32_t key = mix(a.s.seed + mix(static_cast<uint32_t>(r.step) + mix(static_cast<uint32_t>(a.t.first + t))));
  const uint32_t pair = (static_cast<uint32_t>(base >> 1) + key) + 4 * threadIdx.x;
  u32x2_t nm = {0, 0}, nr = {0, 0};
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    float u0, u1;
    mix_chances(pair + k / 2, &u0, &u1);
    const float lo = root_code_value(root[k] * ir, u0, v[k] > 0.0f);
    const float hi = root_code_value(root[k + 1] * ir, u1, v[k + 1] > 0.0f);
    // m: at most 448 (1 + 2^-22), which rounds to 448
    if (k & 2) {
      nm[k >> 2] = __builtin_amdgcn_cvt_pk_fp8_f32(m[k] * im, m[k + 1] * im, nm[k >> 2], true);
      nr[k >> 2] = __builtin_amdgcn_cvt_pk_fp8_f32(lo, hi, nr[k >> 2], true);
    } else {
      nm[k >> 2] = __builtin_amdgcn_cvt_pk_fp8_f32(m[k] * im, m[k + 1] * im, nm[k >> 2], false);
      nr[k >> 2] = __builtin_amdgcn_cvt_pk_fp8_f32(lo, hi, nr[k >> 2], false);
    }
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {  // a group that is stored as zeros, or holds a NaN or an infinity
    nm[q] = im > 0.0f ? nm[q] : 0u;
    nr[q] = ir > 0.0f ? nr[q] : 0u;
  }
  store_codes<FULL>(mc, i, left, nm);
  store_codes<FULL>(rc, i, left, nr);
  if (any && (threadIdx.x & 15) == 0) {
    ms[group] = sm2;
    rs[group] = sr2;
  }
}

template <int DW, int DG, int K>
__global__ __launch_bounds__(kThreads) void adamw8_kernel(AdamwArgs<kPtrs8, K> a) {
  const int t = find_tensor(a.t, blockIdx.x);
  const int64_t n = a.t.size[t], base = static_cast<int64_t>(blockIdx.x - a.t.start[t]) * kChunk8;
  const Scalars r = load_scalars(a.s);
  if (base + kChunk8 <= n) {
    adamw8_chunk<DW, DG, true>(a, t, base, n, r);
  } else {
    adamw8_chunk<DW, DG, false>(a, t, base, n, r);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
muon_status make_scalars(const muon_adamw_config* cfg, AdamwScalars* s) {
  if (cfg == nullptr) return MUON_ERR_INVALID_ARG;
  if (!isfinite(cfg->lr) || !isfinite(cfg->weight_decay) || !isfinite(cfg->eps)) return MUON_ERR_INVALID_ARG;
  if (!(cfg->beta1 >= 0.0) || !(cfg->beta1 < 1.0) || !(cfg->beta2 >= 0.0) || !(cfg->beta2 < 1.0))
    return MUON_ERR_INVALID_ARG;
  if (!(static_cast<float>(cfg->eps) >= 0x1p-126f)) return MUON_ERR_INVALID_ARG;  // its reciprocal is finite
  if (cfg->step_dev == nullptr && cfg->step < 1) return MUON_ERR_INVALID_ARG;
  memset(s, 0, sizeof(*s));
  s->lr = static_cast<float>(cfg->lr);
  s->wd = static_cast<float>(cfg->weight_decay);
  s->eps = static_cast<float>(cfg->eps);
  if (!isfinite(s->lr) || !isfinite(s->wd) || !isfinite(s->eps)) return MUON_ERR_INVALID_ARG;
  s->beta1 = cfg->beta1;
  s->beta2 = cfg->beta2;
  s->b1 = static_cast<float>(cfg->beta1);
  s->b2 = static_cast<float>(cfg->beta2);
  s->ob1 = static_cast<float>(1.0 - cfg->beta1);  // rounded once: 1 - (float)beta2 is off by 1e-5
  s->ob2 = static_cast<float>(1.0 - cfg->beta2);
  s->step = cfg->step;
  s->step_dev = cfg->step_dev;
  s->grad_scale = cfg->grad_scale;
  s->seed = cfg->seed;
  // The 8-bit step's denominator c2 root + eps, c2 at most 1 / sqrt(1 - b2): with a root
  // that is off by 2^-64 at most (root_nearest) its relative error is 2^-26 or less
  // from this eps on (1.2e-10 for b2 = 0.999).
  s->small_eps = cfg->eps < 0x1p-38 / sqrt(1.0 - cfg->beta2);
  if (cfg->step_dev == nullptr) {
    const double left = 1.0 - pow(cfg->beta1, static_cast<double>(cfg->step));
    s->c1 = static_cast<float>(1.0 / left);
    s->lr1 = static_cast<float>(s->lr / left);
    s->wd1 = static_cast<float>(s->wd * left);
    s->c2 = static_cast<float>(1.0 / sqrt(1.0 - pow(cfg->beta2, static_cast<double>(cfg->step))));
  }
  return MUON_OK;
}

// Sizes in range, pointer arrays present and distinct, types known.
muon_status check_lists(int tensors, const int64_t* sizes, const void* const* const* arrays, int narrays,
                        muon_dtype w_dtype, muon_dtype g_dtype, int chunk) {
  if (tensors < 1 || sizes == nullptr) return MUON_ERR_INVALID_ARG;
  for (int i = 0; i < narrays; ++i) {
    if (arrays[i] == nullptr) return MUON_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (arrays[i] == arrays[j]) return MUON_ERR_INVALID_ARG;
  }
  for (int i = 0; i < tensors; ++i)
    if (sizes[i] < 0 || sizes[i] / chunk >= (1 << 23)) return MUON_ERR_INVALID_ARG;  // over any device's memory
  const muon_dtype types[2] = {w_dtype, g_dtype};
  for (muon_dtype d : types)
    if (d != MUON_F32 && d != MUON_BF16 && d != MUON_F16) return MUON_ERR_INVALID_ARG;
  if (w_dtype == MUON_F16) return MUON_ERR_UNSUPPORTED;
  for (int i = 0; i < tensors; ++i)
    for (int j = 0; j < narrays; ++j)
      if (sizes[i] > 0 && arrays[j][i] == nullptr) return MUON_ERR_INVALID_ARG;
  return MUON_OK;
}

// The next launch's tensors from `at` on: as many as fit and as keep the
// blocks under the grid's limit.  Returns the blocks.
template <int P, int K>
uint32_t fill_lists(Lists<P, K>* t, int tensors, const int64_t* sizes, const void* const* const* arrays, int at,
                    int chunk) {
  t->first = at;
  t->count = 0;
  uint32_t blocks = 0;
  t->start[0] = 0;
  while (t->count < K && at + t->count < tensors) {
    const int c = t->count;
    const int64_t n = sizes[at + c];
    const uint32_t b = static_cast<uint32_t>((n + chunk - 1) / chunk);
    if (c > 0 && blocks + b > (1u << 23)) break;
    blocks += b;
    t->size[c] = n;
    for (int j = 0; j < P; ++j) t->ptr[j][c] = const_cast<void*>(arrays[j][at + c]);
    t->start[++t->count] = blocks;
  }
  return blocks;
}

// A launch of `kernel<DW, DG, K>`.
#define ADAMW_TYPES(kernel, K, args, blocks, w, g, s)                                                     \
  do {                                                                                                    \
    const dim3 grid_(blocks), block_(kThreads);                                                           \
    if ((w) == MUON_F32) {                                                                                \
      if ((g) == MUON_F32) hipLaunchKernelGGL((kernel<kF32, kF32, K>), grid_, block_, 0, s, args);        \
      else if ((g) == MUON_BF16) hipLaunchKernelGGL((kernel<kF32, kBF16, K>), grid_, block_, 0, s, args); \
      else hipLaunchKernelGGL((kernel<kF32, kF16, K>), grid_, block_, 0, s, args);                        \
    } else {                                                                                              \
      if ((g) == MUON_F32) hipLaunchKernelGGL((kernel<kBF16, kF32, K>), grid_, block_, 0, s, args);       \
      else if ((g) == MUON_BF16) hipLaunchKernelGGL((kernel<kBF16, kBF16, K>), grid_, block_, 0, s, args);\
      else hipLaunchKernelGGL((kernel<kBF16, kF16, K>), grid_, block_, 0, s, args);                       \
    }                                                                                                     \
  } while (0)

double element_bytes(muon_dtype w, muon_dtype g, double state_bytes) {
  return (w == MUON_F32 ? 8.0 : 4.0) + (g == MUON_F32 ? 4.0 : 2.0) + state_bytes;
}

// The launches of one call; `launch(args, blocks, stream)` for each.
template <int P, int K, class Launch>
muon_status run_lists(const AdamwScalars& scalars, int tensors, const int64_t* sizes, const void* const* const* arrays,
                      int chunk, double element, const char* kernel, const char* role, hipStream_t s, Launch&& launch) {
  AdamwArgs<P, K> a;
  a.s = scalars;
  for (int at = 0; at < tensors;) {
    const uint32_t blocks = fill_lists(&a.t, tensors, sizes, arrays, at, chunk);
    at += a.t.count;
    if (blocks == 0) continue;  // empty tensors only
    double elems = 0.0;
    for (int i = 0; i < a.t.count; ++i) elems += static_cast<double>(a.t.size[i]);
    const hipError_t err = traced_launch(s, kernel, role, 0.0, elems * element, [&] {
      launch(a, blocks);
      return hipGetLastError();
    });
    if (err != hipSuccess) return MUON_ERR_HIP;
  }
  return MUON_OK;
}

template <int K>
muon_status run32(const AdamwScalars& scalars, int tensors, const int64_t* sizes, const void* const* const* arrays,
                  muon_dtype w, muon_dtype g, hipStream_t s) {
  return run_lists<kPtrs32, K>(scalars, tensors, sizes, arrays, kChunk32, element_bytes(w, g, 16.0), "adamw_kernel",
                               "adamw", s, [&](const AdamwArgs<kPtrs32, K>& a, uint32_t blocks) {
                                 ADAMW_TYPES(adamw_kernel, K, a, blocks, w, g, s);
                               });
}

template <int K>
muon_status run8(const AdamwScalars& scalars, int tensors, const int64_t* sizes, const void* const* const* arrays,
                 muon_dtype w, muon_dtype g, hipStream_t s) {
  return run_lists<kPtrs8, K>(scalars, tensors, sizes, arrays, kChunk8, element_bytes(w, g, 4.0 + 16.0 / kGroup),
                              "adamw8_kernel", "adamw8", s, [&](const AdamwArgs<kPtrs8, K>& a, uint32_t blocks) {
                                ADAMW_TYPES(adamw8_kernel, K, a, blocks, w, g, s);
                              });
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

void muon_adamw_config_init(muon_adamw_config* cfg) {
  if (cfg == nullptr) return;
  memset(cfg, 0, sizeof(*cfg));
  cfg->lr = 1e-3;
  cfg->beta1 = 0.9;
  cfg->beta2 = 0.999;
  cfg->eps = 1e-8;
  cfg->step = 1;
}

muon_status muon_adamw_step(int tensors, const int64_t* sizes, void* const* W, muon_dtype w_dtype, void* const* M,
                            void* const* V, const void* const* G, muon_dtype g_dtype, const muon_adamw_config* cfg,
                            void* stream) {
  const void* const* arrays[4] = {W, G, M, V};
  muon_status st = check_lists(tensors, sizes, arrays, 4, w_dtype, g_dtype, kChunk32);
  if (st != MUON_OK) return st;
  AdamwScalars scalars;
  st = make_scalars(cfg, &scalars);
  if (st != MUON_OK) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return tensors <= kFew ? run32<kFew>(scalars, tensors, sizes, arrays, w_dtype, g_dtype, s)
                         : run32<many_tensors(kPtrs32)>(scalars, tensors, sizes, arrays, w_dtype, g_dtype, s);
}

muon_status muon_adamw8_step(int tensors, const int64_t* sizes, void* const* W, muon_dtype w_dtype,
                             const muon_adamw8_state* state, const void* const* G, muon_dtype g_dtype,
                             const muon_adamw_config* cfg, void* stream) {
  if (state == nullptr) return MUON_ERR_INVALID_ARG;
  const void* const* arrays[6] = {W, G, state->m_codes, state->m_scales, state->r_codes, state->r_scales};
  muon_status st = check_lists(tensors, sizes, arrays, 6, w_dtype, g_dtype, kChunk8);
  if (st != MUON_OK) return st;
  AdamwScalars scalars;
  st = make_scalars(cfg, &scalars);
  if (st != MUON_OK) return st;
  // weight8's quotients in fp32: lr c1, largest at t = 1, and 1 / eps in the normal range
  if (!isfinite(static_cast<float>(scalars.lr / (1.0 - cfg->beta1))) || !(scalars.eps <= 0x1p126f))
    return MUON_ERR_INVALID_ARG;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return tensors <= kFew ? run8<kFew>(scalars, tensors, sizes, arrays, w_dtype, g_dtype, s)
                         : run8<many_tensors(kPtrs8)>(scalars, tensors, sizes, arrays, w_dtype, g_dtype, s);
}

}  // extern "C"

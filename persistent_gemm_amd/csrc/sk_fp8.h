// Device helpers of the fp32-block-scaled E4M3 operators: the scale of a block, correctly
// rounded codes, lane reductions, and loads of rows that are aligned only to their elements.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sk {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
// The same bytes at any element's address: a row of an odd length starts anywhere.
typedef u32x4 u32x4_any __attribute__((aligned(2)));

// A launch with its arguments given by address: the triple-chevron form passes them through a call-configuration stack,
// 0.2 us of the 2.4 that a launch takes the host.
template <class... P>
inline hipError_t launch(void (*kernel)(P...), dim3 grid, int threads, hipStream_t s, P... a) {
  void* args[] = {(void*)&a...};
  const hipError_t e = hipLaunchKernel((const void*)kernel, grid, dim3((unsigned)threads), args, 0, s);
  if (e != hipSuccess) (void)hipGetLastError();
  return e;
}

constexpr int kBlock = 128;              // elements that share a scale
constexpr float kScaleMin = 0x1p-126f;   // the smallest scale (an empty or all-zero block has it)
constexpr uint32_t kAbs = 0x7fffffffu;

__device__ __forceinline__ float bits_f(uint32_t u) { return __uint_as_float(u); }
__device__ __forceinline__ uint32_t f_bits(float f) { return __float_as_uint(f); }
__device__ __forceinline__ float bf16_lo(uint32_t w) { return bits_f(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return bits_f(w & 0xffff0000u); }

// bf16 to nearest-even of two floats, packed.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  typedef float f2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{a, b}), b2));
}

// Eight consecutive elements of a row as they lie in memory: what a load in flight occupies.
template <class T>
struct Raw8 {
  u32x4 w[sizeof(T) / 2];
};

// Elements col .. col + 7 of a row of D.  Past D - 8 the last eight are loaded instead, to be moved into place by
// settle8 once they are needed: a branch around the load would make every later load wait for this one.  The
// column is an unsigned 32-bit offset from an address that all lanes share.  SHORT: D < 8, element by element.
template <bool SHORT, class T>
__device__ __forceinline__ Raw8<T> load_raw8(const T* __restrict__ row, int col, int D) {
  Raw8<T> r;
  if constexpr (!SHORT) {
    const T* const p = row + (uint32_t)min(col, D - 8);
#pragma unroll
    for (unsigned i = 0; i < sizeof(T) / 2; ++i) r.w[i] = *(const u32x4_any*)(p + 8 / (sizeof(T) / 2) * i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool in = col + i < D;
      if constexpr (sizeof(T) == 4) {
        r.w[i / 4][i % 4] = in ? f_bits(row[col + i]) : 0u;
      } else {
        const uint32_t x = in ? (uint32_t)row[col + i] : 0u;
        if (i % 2 == 0) r.w[0][i / 2] = x;
        else r.w[0][i / 2] |= x << 16;
      }
    }
  }
  return r;
}

// The loaded elements moved to their places, zeros behind the row's end.
template <bool SHORT, class T>
__device__ __forceinline__ void settle8(Raw8<T>& r, int col, int D) {
  if constexpr (!SHORT) {
    const int s = col - (D - 8);     // how far back they were taken
    if (s > 0) {
      constexpr int W = 2 * sizeof(T);   // words
      uint32_t x[W];
#pragma unroll
      for (int i = 0; i < W; ++i) x[i] = s < 8 ? r.w[i / 4][i % 4] : 0u;
      constexpr int PER = 4 / sizeof(T);   // elements of a word
#pragma unroll
      for (int h = 4; h >= PER; h /= 2)
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] = s & h ? (i + h / PER < W ? x[i + h / PER] : 0u) : x[i];
      if constexpr (PER == 2) {
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] = s & 1 ? (x[i] >> 16) | (i + 1 < W ? x[i + 1] << 16 : 0u) : x[i];
      }
#pragma unroll
      for (int i = 0; i < W; ++i) r.w[i / 4][i % 4] = x[i];
    }
  }
}

template <class T>
__device__ __forceinline__ float raw_at(const Raw8<T>& r, int i) {
  if constexpr (sizeof(T) == 4) return bits_f(r.w[i / 4][i % 4]);
  else return i % 2 ? bf16_hi(r.w[0][i / 2]) : bf16_lo(r.w[0][i / 2]);
}

// Stores the first n of eight values, rounded to the element type.
__device__ __forceinline__ void store8(uint16_t* __restrict__ p, int n, const float (&x)[8]) {
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
  if (n >= 8) {
    *(u32x4_any*)p = v;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
  }
}
__device__ __forceinline__ void store8(float* __restrict__ p, int n, const float (&x)[8]) {
  if (n >= 8) {
    *(u32x4_any*)p = u32x4{f_bits(x[0]), f_bits(x[1]), f_bits(x[2]), f_bits(x[3])};
    *(u32x4_any*)(p + 4) = u32x4{f_bits(x[4]), f_bits(x[5]), f_bits(x[6]), f_bits(x[7])};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = x[i];
  }
}

// x as the element type holds it.
template <class T>
__device__ __forceinline__ float rounded(float x);
template <>
__device__ __forceinline__ float rounded<float>(float x) { return x; }
template <>
__device__ __forceinline__ float rounded<uint16_t>(float x) { return bf16_lo(pack_bf16(x, x)); }

// ---------------------------------------------------------------- reductions

// Lane i of a row of 16 lanes gets lane (i + N) % 16 of it.
template <int N>
__device__ __forceinline__ uint32_t row_rotate(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x120 + N, 0xf, 0xf, true);
}

// The largest of 16 lanes' values, in each of them.  Magnitudes of floats are
// compared as integers, which orders finite < infinity < NaN: a block that holds
// an infinity or a NaN keeps it, where a float maximum would drop the NaN.
__device__ __forceinline__ uint32_t max16(uint32_t x) {
  x = max(x, row_rotate<8>(x));
  x = max(x, row_rotate<4>(x));
  x = max(x, row_rotate<2>(x));
  return max(x, row_rotate<1>(x));
}

template <int N>
__device__ __forceinline__ float row_rotated(float x) { return bits_f(row_rotate<N>(f_bits(x))); }
template <int N>
__device__ __forceinline__ double row_rotated(double x) {
  return __hiloint2double((int)row_rotate<N>((uint32_t)__double2hiint(x)), (int)row_rotate<N>((uint32_t)__double2loint(x)));
}

// The sum over a wave, in every lane: rotations within 16 lanes, then across them.  The order is fixed.
template <class T>
__device__ __forceinline__ T wave_sum(T x) {
  x += row_rotated<8>(x);
  x += row_rotated<4>(x);
  x += row_rotated<2>(x);
  x += row_rotated<1>(x);
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

// ---------------------------------------------------------------- scales and codes

// How a block's elements become codes: its scale s, and what the codes' rounding needs.
struct BlockScale {
  float s;    // what is stored
  float r;    // about 1 / s
  float c;    // Coder<float>: a large multiple of r; Coder<uint16_t>: the low part of 1 / s
};

// s = amax / 448 rounded once, at least 2^-126; NaN where the block holds an infinity or a NaN.
// (The quotient's first guess is within an ulp, and one residual step of a division by a constant
// whose reciprocal is correctly rounded gives the nearest value.)  *residual: the sign of
// amax - 448 s is the sign of the scale's own rounding, 0 where s is exact or the smallest.
__device__ __forceinline__ float block_scale(uint32_t amax_bits, float* residual) {
  const float amax = bits_f(amax_bits);
  constexpr float kInv = 1.0f / 448.0f;
  float s = amax * kInv;
  s = __builtin_fmaf(__builtin_fmaf(-s, 448.0f, amax), kInv, s);
  const bool small = s < kScaleMin;
  s = small ? kScaleMin : s;
  *residual = small ? 0.0f : __builtin_fmaf(-s, 448.0f, amax);
  return s;
}

// 1 / s, within an ulp or so (s is a normal number here).
__device__ __forceinline__ float reciprocal(float s) {
  const float r = __builtin_amdgcn_rcpf(s);
  return __builtin_fmaf(__builtin_fmaf(-s, r, 1.0f), r, r);
}

// Codes of the exact quotient x / s, to nearest, ties to even.  A quotient rounded to fp32
// first would be rounded twice: x / s often lies on the border between two codes (448 x / amax
// is a short fraction) or within 2^-28 of it, and both would come out as the border.
template <class T>
struct Coder;

// fp32: t is the quotient to five bits, which holds every code and every border, and the sign of
// x - t s (one fma, so the sign is exact) says on which side of t the quotient lies.  t is moved that way
// by far less than the distance to the next border and far more than an ulp, and the conversion rounds it.
// The difference is at least 2^-29 |t| s where it is not 0, which is less than the smallest fp32 for s below 2^-110: where
// a wave has a scale below 2^-96, such blocks' values and scales are first multiplied by 2^64.  (As a branch: one more
// product for every value, 8192x4096 bf16, takes the norm to fp8 from 26.1 to 27.1 us, the branch to 25.8.)
template <>
struct Coder<float> {
  static __device__ __forceinline__ BlockScale scale(uint32_t amax_bits) {
    BlockScale b;
    float residual;
    b.s = block_scale(amax_bits, &residual);
    b.r = reciprocal(b.s);
    // x - t s times this is at least 2 |t|, so clamped to 2^-10 a step of its sign for every t of the codes' range
    b.c = b.r * 0x1p30f;
    return b;
  }
  static __device__ __forceinline__ bool small(const BlockScale& b) { return b.s < 0x1p-96f; }
  // What to multiply a small block's values by; its scale is.
  static __device__ __forceinline__ float lift(BlockScale& b) {
    const bool low = small(b);
    const float up = low ? 0x1p64f : 1.0f;
    b.s *= up;
    b.r *= low ? 0x1p-64f : 1.0f;
    b.c = b.r * 0x1p30f;
    return up;
  }
  // Values of one block, multiplied where it is small, in units of its scale.
  template <int N>
  static __device__ __forceinline__ void nudge_lifted(float (&v)[N], const BlockScale& b) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float q = v[k] * b.r;
      const float t = bits_f((f_bits(q) + 0x40000u) & 0xfff80000u);
      const float e = __builtin_fmaf(-t, b.s, v[k]);
      const float n = __builtin_amdgcn_fmed3f(e * b.c, -0x1p-10f, 0x1p-10f);
      v[k] = __builtin_fmaf(__builtin_fabsf(t), n, t);
    }
  }
  template <int N>
  static __device__ __forceinline__ void nudge(float (&v)[N], BlockScale b) {
    if (__builtin_expect(__any(small(b)), 0)) {
      const float up = lift(b);
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] *= up;
    }
    nudge_lifted(v, b);
  }
};

// bf16: x = X 2^a and amax = Y 2^b with X, Y < 2^8, so 448 x / amax is a border or at least 2^-13 away from
// it, and only the scale's own rounding can then move x / s off the border: its sign is known.  The
// reciprocal is taken that much (2^-20) too large or too small where s is not exact; where it is, x / s
// is computed exactly where it is short: 1 / s in two parts, the first of 16 bits (its product with x is exact).
template <>
struct Coder<uint16_t> {
  static __device__ __forceinline__ BlockScale scale(uint32_t amax_bits) {
    BlockScale b;
    float residual;
    b.s = block_scale(amax_bits, &residual);
    const float r = reciprocal(b.s);
    b.r = bits_f(f_bits(r) & 0xffffff00u);
    b.c = r * __builtin_fmaf(-b.s, b.r, 1.0f);
    // amax > 448 s: the scale was rounded down, so x / s lies beyond 448 x / amax
    b.c += residual > 0.0f ? r * 0x1p-20f : residual < 0.0f ? r * -0x1p-20f : 0.0f;
    return b;
  }
  template <int N>
  static __device__ __forceinline__ void nudge(float (&v)[N], const BlockScale& b) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = __builtin_fmaf(v[k], b.c, v[k] * b.r);
  }
};

constexpr uint32_t kNanCodes = 0x7f7f7f7fu;

// Four codes of values already in units of the scale s; a block whose scale is NaN has NaN codes
// (chosen here: the steps above do not carry every NaN through).
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float s) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return s != s ? kNanCodes : (uint32_t)w;
}

}  // namespace sk

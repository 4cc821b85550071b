// 4-bit codes of a weight with a 16-bit scale (and a zero point) for each group along a row, and the values they
// stand for:
//
//   without zero points   s = max|w| / 7,              q = 8 + w / s        (codes 1 .. 15)
//   with them             s = (hi - lo) / 15,          z = -lo / s,  q = z + w / s,   hi = max(w, 0), lo = min(w, 0)
//
// each quotient to nearest, ties to even, codes and zero points held to 0 .. 15.  s is rounded to its type (and at least its
// smallest normal number) before it divides.  A group with an infinity or a NaN, or whose scale is beyond its type, has a NaN
// scale, and codes and a zero point of 0.

#include "sk_experts.h"

namespace sk {

namespace {

// w / s to the nearest whole number, ties to even.  The fp32 quotient may have been rounded onto a border between two
// numbers: the sign of w - border s (one fma, exact in sign) then says on which side the exact one lies.
__device__ __forceinline__ float nearest(float w, float s) {
  const float v = w / s;
  float r = rintf(v);
  const float border = r < v ? r + 0.5f : r - 0.5f;      // the one next to v
  if (v == border) {
    const float e = __builtin_fmaf(-border, s, w);
    if (e > 0.0f) r = border + 0.5f;
    if (e < 0.0f) r = border - 0.5f;
  }
  return r;
}

// 8 elements to a thread, G / 8 threads to a group; a workgroup takes 256 / (G / 8) consecutive rows of one group column, so
// that its scales are one stretch.
template <class T, class S, int G, bool ZERO>
__global__ __launch_bounds__(256) void sk_quantize4(Quant4Args a) {
  constexpr int L = G / 8, ROWS = 256 / L;
  const int groups = a.K / G, l = threadIdx.x % L;
  const int64_t blocks_n = (a.N + ROWS - 1) / ROWS;
  const int64_t b = blockIdx.x;
  const int col = (int)(b % groups);
  const int64_t rb = b / groups;
  const int e = (int)(rb / blocks_n);
  const int n = (int)(rb % blocks_n) * ROWS + (int)threadIdx.x / L;
  if (n >= a.N) return;
  const int64_t row = (int64_t)e * a.N + n;
  const Vec8<T> x = load8<false>((const T*)a.w + row * a.K, col * G + l * 8, a.K);
  constexpr float tiny = std::is_same_v<S, _Float16> ? 0x1p-14f : 0x1p-126f;
  float hi = 0.0f, lo = 0.0f;
  uint32_t mag = 0;                       // (as integers a NaN is the largest)
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    hi = fmaxf(hi, x.v[i]);
    lo = fminf(lo, x.v[i]);
    mag = max(mag, f_bits(x.v[i]) & kAbs);
  }
#pragma unroll
  for (int d = 1; d < L; d *= 2) {
    hi = fmaxf(hi, __shfl_xor(hi, d));
    lo = fminf(lo, __shfl_xor(lo, d));
    mag = max(mag, (uint32_t)__shfl_xor((int)mag, d));
  }
  float s = ZERO ? (hi - lo) / 15.0f : bits_f(mag) / 7.0f;
  S stored;
  store_elem(&stored, s);
  s = fmaxf(load_elem(&stored), tiny);
  const bool bad = mag >= 0x7f800000u || s == __builtin_inff();
  store_elem(&stored, bad ? __builtin_nanf("") : s);
  const float z = ZERO ? fminf(fmaxf(nearest(-lo, s), 0.0f), 15.0f) : 8.0f;
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = fminf(fmaxf(nearest(x.v[i], s) + z, 0.0f), 15.0f);
    codes |= (bad ? 0u : (uint32_t)q) << (4 * i);
  }
  *(uint32_t*)(a.q + row * (a.K / 2) + col * (G / 2) + l * 4) = codes;
  if (l == 0) {
    const int64_t at = ((int64_t)e * groups + col) * a.N + n;
    ((S*)a.scale)[at] = stored;
    if (ZERO) a.zero[at] = bad ? (uint8_t)0 : (uint8_t)z;
  }
}

// Eight codes to a thread.
template <class S>
__global__ __launch_bounds__(256) void sk_dequantize4(Quant4Args a) {
  const int per_row = a.K / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = i / per_row;
  if (row >= (int64_t)a.E * a.N) return;
  const int c = (int)(i - row * per_row);
  const int e = (int)(row / a.N), n = (int)(row - (int64_t)e * a.N);
  const int groups = a.K / a.group;
  const int64_t at = ((int64_t)e * groups + c * 8 / a.group) * a.N + n;
  const float s = load_elem((const S*)a.scale + at);
  const float z = a.zero ? (float)a.zero[at] : 8.0f;
  const uint32_t d = *(const uint32_t*)(a.q + row * (a.K / 2) + c * 4);
  float x[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = s * ((float)(d >> (4 * k) & 15u) - z);
  put8((S*)a.out + row * a.K + c * 8, 8, x);
}

template <class T, class S, bool ZERO>
hipError_t by_group(const Quant4Args& a, hipStream_t s) {
  auto go = [&](auto g) {
    constexpr int G = decltype(g)::value;
    const int64_t blocks = ((int64_t)a.N + 256 / (G / 8) - 1) / (256 / (G / 8)) * a.E * (a.K / G);
    if (blocks > 0x7fffffff) return hipErrorInvalidValue;
    return launch(sk_quantize4<T, S, G, ZERO>, dim3((unsigned)blocks), 256, s, a);
  };
  if (a.group == 32) return go(std::integral_constant<int, 32>{});
  if (a.group == 64) return go(std::integral_constant<int, 64>{});
  return go(std::integral_constant<int, 128>{});
}
template <class T, class S>
hipError_t by_zero(const Quant4Args& a, hipStream_t s) {
  return a.zero ? by_group<T, S, true>(a, s) : by_group<T, S, false>(a, s);
}

}  // namespace

hipError_t launch_quantize_w4(const Quant4Args& a, int elem, bool f16, hipStream_t s) {
  if (elem == SK_ELEM_BF16) return f16 ? by_zero<BfElem, _Float16>(a, s) : by_zero<BfElem, BfElem>(a, s);
  if (elem == SK_ELEM_F16) return f16 ? by_zero<_Float16, _Float16>(a, s) : by_zero<_Float16, BfElem>(a, s);
  return f16 ? by_zero<float, _Float16>(a, s) : by_zero<float, BfElem>(a, s);
}

hipError_t launch_dequantize_w4(const Quant4Args& a, bool f16, hipStream_t s) {
  const int64_t blocks = ((int64_t)a.E * a.N * (a.K / 8) + 255) / 256;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  return f16 ? launch(sk_dequantize4<_Float16>, dim3((unsigned)blocks), 256, s, a)
             : launch(sk_dequantize4<BfElem>, dim3((unsigned)blocks), 256, s, a);
}

}  // namespace sk

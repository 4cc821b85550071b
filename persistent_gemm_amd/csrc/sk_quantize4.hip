// 4-bit codes of a weight with a 16-bit scale (and a zero point) for each group along a row, and the values they
// stand for:
//
//   without zero points   s = max|w| / 7,              q = 8 + w / s        (codes 1 .. 15)
//   with them             s = (hi - lo) / 15,          z = -lo / s,  q = z + w / s,   hi = max(w, 0), lo = min(w, 0)
//
// each quotient to nearest, ties to even, codes and zero points held to 0 .. 15.  s is rounded to its type (and at least its
// smallest normal number) before it divides; the difference hi - lo and the quotient are fp32's before that, so that next to the border
// between two of its type's numbers s may be the other one (about one group in 10^5 of an fp32 weight; the codes fit the s that is
// stored all the same).  A group with an infinity or a NaN, or whose scale is beyond its type, has a NaN scale, and codes and a zero point
// of 0.

#include "sk_experts.h"

namespace sk {

namespace {

// w / s to the nearest whole number, ties to even, with r about 1 / s.  16-bit w and s: the quotient is a border between two
// numbers or at least 2^-14 from one, so the fp32 quotient decides (a product, corrected by its residual, is the nearest one).
// fp32 w: the sign of w - border s (one fma, exact in sign) says on which side of the border next to it the quotient lies.
template <class T>
__device__ __forceinline__ float nearest(float w, float s, float r) {
  const float v = w * r;
  if constexpr (sizeof(T) == 2) {
    return rintf(__builtin_fmaf(__builtin_fmaf(-v, s, w), r, v));
  } else {
    const float border = floorf(v) + 0.5f;
    const float e = __builtin_fmaf(-border, s, w) * r;
    return rintf(border + __builtin_amdgcn_fmed3f(e * 0x1p30f, -0x1p-10f, 0x1p-10f));
  }
}

// 8 elements to a thread, G / 8 threads to a group, a wave to 512 consecutive elements of a row; a workgroup takes those of ROWS rows, a
// quarter to each wave, and stores their scales, which lie row by row, in stretches.  Bound by memory: 8192 x 8192 bf16 37.5 us from
// memory (4.5 TB/s; with a division for each element and 256 bytes of a row at a time nearly twice that).
template <class T, class S, int G, bool ZERO, int ROWS>
__global__ __launch_bounds__(256) void sk_quantize4(Quant4Args a) {
  constexpr int L = G / 8, PER = 512 / G;        // lanes of a group; groups of a wave's stretch
  constexpr int kRows4 = ROWS, kAhead4 = ROWS / 4 < 4 ? ROWS / 4 : 4;     // (rows whose loads are under way together)
  __shared__ S scales[PER][kRows4];
  __shared__ uint8_t zeros[PER][kRows4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int cols = (a.K + 511) / 512, rows_of = (a.N + kRows4 - 1) / kRows4, groups = a.K / G;
  const int col = (int)(blockIdx.x % (unsigned)cols) * 512;
  const int rb = (int)(blockIdx.x / (unsigned)cols), e = rb / rows_of, n0 = (rb - e * rows_of) * kRows4;
  const int k = col + lane * 8;
  const bool in = k < a.K;
  constexpr float tiny = std::is_same_v<S, _Float16> ? 0x1p-14f : 0x1p-126f;
  const T* const w = (const T*)a.w + ((int64_t)e * a.N + n0) * a.K;
  uint8_t* const q = a.q + ((int64_t)e * a.N + n0) * (a.K / 2);
  const int have = min(kRows4, a.N - n0);
  using R = std::conditional_t<sizeof(T) == 4, float, uint16_t>;
  for (int r0 = wave * (kRows4 / 4); r0 < min((wave + 1) * (kRows4 / 4), have); r0 += kAhead4) {
    Raw8<R> raw[kAhead4];
#pragma unroll
    for (int i = 0; i < kAhead4; ++i)
      raw[i] = load_raw8<false>((const R*)w + (int64_t)min(r0 + i, have - 1) * a.K, in ? k : 0, a.K);
#pragma unroll
    for (int i = 0; i < kAhead4; ++i) {
      const int n = r0 + i;
      const Vec8<T> x = unpack8<T>(raw[i]);
      float hi = 0.0f, lo = 0.0f;
      uint32_t mag = 0;                       // (as integers a NaN is the largest)
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if constexpr (ZERO) {
          hi = fmaxf(hi, x.v[c]);
          lo = fminf(lo, x.v[c]);
        }
        mag = max(mag, f_bits(x.v[c]) & kAbs);
      }
#pragma unroll
      for (int d = 1; d < L; d *= 2) {
        if constexpr (ZERO) {
          hi = fmaxf(hi, __shfl_xor(hi, d));
          lo = fminf(lo, __shfl_xor(lo, d));
        }
        mag = max(mag, (uint32_t)__shfl_xor((int)mag, d));
      }
      float s = ZERO ? (hi - lo) / 15.0f : bits_f(mag) / 7.0f;
      if constexpr (ZERO && !std::is_same_v<T, _Float16>) {
        // A difference beyond fp32, whose scale is not: of halves.  (A branch that the wave hardly ever takes; as a choice between the
        // two 8192 x 8192 bf16 took 38.8 us and not 37.6.)
        if (__builtin_expect(__ballot(s == __builtin_inff()) != 0, 0)) {
          const float half = (0.5f * hi - 0.5f * lo) / 15.0f;
          s = s == __builtin_inff() ? 2.0f * half : s;
        }
      }
      S stored;
      store_elem(&stored, s);
      s = fmaxf(load_elem(&stored), tiny);
      const bool bad = mag >= 0x7f800000u || s == __builtin_inff();
      store_elem(&stored, bad ? __builtin_nanf("") : s);
      const float r = reciprocal(s);
      // (the difference of two 16-bit numbers has more bits: -lo is one of them)
      const float z = ZERO ? fminf(fmaxf(nearest<T>(-lo, s, r), 0.0f), 15.0f) : 8.0f;
      uint32_t even = 0, odd = 0;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float y = __builtin_amdgcn_fmed3f(nearest<T>(x.v[c], s, r) + z, 0.0f, 15.0f);
        uint32_t& to = c % 2 ? odd : even;
        to = __builtin_amdgcn_cvt_pk_u8_f32(y, c / 2, to);
      }
      if (in && n < have) {
        *(uint32_t*)(q + (int64_t)n * (a.K / 2) + k / 2) = bad ? 0u : even | odd << 4;
        if (lane % L == 0) {
          scales[lane / L][n] = stored;
          if (ZERO) zeros[lane / L][n] = bad ? (uint8_t)0 : (uint8_t)z;
        }
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < PER * kRows4; i += 256) {
    const int g = i / kRows4, n = i % kRows4;
    if (col / G + g < groups && n < have) {
      const int64_t at = ((int64_t)e * groups + col / G + g) * a.N + n0 + n;
      ((S*)a.scale)[at] = scales[g][n];
      if (ZERO) a.zero[at] = zeros[g][n];
    }
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
hipError_t by_group(const Quant4Args& a, int cus, hipStream_t s) {
  auto go = [&](auto g) {
    constexpr int G = decltype(g)::value;
    auto blocks = [&](int rows) { return ((int64_t)a.N + rows - 1) / rows * a.E * ((a.K + 511) / 512); };
    // fewer rows to a workgroup where there would not be four to a unit: 515 x 1312 fp32 with zero points 3.4 us against 6.7
    if (blocks(32) < 4 * (int64_t)cus) return launch(sk_quantize4<T, S, G, ZERO, 4>, dim3((unsigned)blocks(4)), 256, s, a);
    if (blocks(32) > 0x7fffffff) return hipErrorInvalidValue;
    return launch(sk_quantize4<T, S, G, ZERO, 32>, dim3((unsigned)blocks(32)), 256, s, a);
  };
  if (a.group == 32) return go(std::integral_constant<int, 32>{});
  if (a.group == 64) return go(std::integral_constant<int, 64>{});
  return go(std::integral_constant<int, 128>{});
}
template <class T, class S>
hipError_t by_zero(const Quant4Args& a, int cus, hipStream_t s) {
  return a.zero ? by_group<T, S, true>(a, cus, s) : by_group<T, S, false>(a, cus, s);
}

}  // namespace

hipError_t launch_quantize_w4(const Quant4Args& a, int elem, bool f16, int cus, hipStream_t s) {
  if (elem == SK_ELEM_BF16) return f16 ? by_zero<BfElem, _Float16>(a, cus, s) : by_zero<BfElem, BfElem>(a, cus, s);
  if (elem == SK_ELEM_F16) return f16 ? by_zero<_Float16, _Float16>(a, cus, s) : by_zero<_Float16, BfElem>(a, cus, s);
  return f16 ? by_zero<float, _Float16>(a, cus, s) : by_zero<float, BfElem>(a, cus, s);
}

hipError_t launch_dequantize_w4(const Quant4Args& a, bool f16, hipStream_t s) {
  const int64_t blocks = ((int64_t)a.E * a.N * (a.K / 8) + 255) / 256;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  return f16 ? launch(sk_dequantize4<_Float16>, dim3((unsigned)blocks), 256, s, a)
             : launch(sk_dequantize4<BfElem>, dim3((unsigned)blocks), 256, s, a);
}

}  // namespace sk

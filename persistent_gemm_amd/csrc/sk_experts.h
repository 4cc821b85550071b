// Element access of the row-wise operators of a layer of experts: bf16, fp16 and fp32.
#pragma once

#include <algorithm>
#include <type_traits>

#include "../../include/sk_gemm.h"
#include "sk_common.h"
#include "sk_fp8.h"

namespace sk {

// A bf16 element (as bits); fp16 and fp32 are _Float16 and float.
struct BfElem {
  uint16_t u;
};

__device__ __forceinline__ float load_elem(const BfElem* p) { return bf16_lo(p->u); }
__device__ __forceinline__ float load_elem(const _Float16* p) { return (float)*p; }
__device__ __forceinline__ float load_elem(const float* p) { return *p; }
__device__ __forceinline__ void store_elem(BfElem* p, float x) { p->u = (uint16_t)pack_bf16(x, x); }
__device__ __forceinline__ void store_elem(_Float16* p, float x) { *p = (_Float16)x; }
__device__ __forceinline__ void store_elem(float* p, float x) { *p = x; }

// Eight elements of a row from column col on, as floats; those behind the row's end are zeros.
template <class T>
struct Vec8 {
  float v[8];
};
template <class T, class R>
__device__ __forceinline__ Vec8<T> unpack8(const Raw8<R>& r) {
  Vec8<T> x;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (std::is_same_v<T, _Float16>) {
      const uint32_t w = r.w[0][i / 2];
      x.v[i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(i % 2 ? w >> 16 : w));
    } else {
      x.v[i] = raw_at(r, i);
    }
  }
  return x;
}
template <bool SHORT, class T>
__device__ __forceinline__ Vec8<T> load8(const T* row, int col, int D) {
  using R = std::conditional_t<sizeof(T) == 4, float, uint16_t>;
  Raw8<R> r = load_raw8<SHORT>((const R*)row, col, D);
  settle8<SHORT>(r, col, D);
  return unpack8<T>(r);
}
// Stores the first n of eight values, rounded to the element type.
__device__ __forceinline__ void put8(BfElem* p, int n, const float (&x)[8]) { store8((uint16_t*)p, n, x); }
__device__ __forceinline__ void put8(float* p, int n, const float (&x)[8]) { store8(p, n, x); }
__device__ __forceinline__ void put8(_Float16* p, int n, const float (&x)[8]) {
  typedef _Float16 h8 __attribute__((ext_vector_type(8)));
  typedef h8 h8_any __attribute__((aligned(2)));
  if (n >= 8) {
    h8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (_Float16)x[i];
    *(h8_any*)p = v;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (_Float16)x[i];
  }
}

}  // namespace sk

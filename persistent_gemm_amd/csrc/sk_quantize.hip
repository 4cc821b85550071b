// The block quantiser: E4M3 codes and fp32 scales of blocks of 128 along a row, or of 128 x 128,
// of a bf16 or fp32 matrix, of its transpose, or of both in one pass over it.
//
//   s = max(fl(max|x| / 448), 2^-126) over the block,   q = E4M3 nearest to x / s, ties to even.
//
// A workgroup takes one 128 x 128 tile: thread (tr, tc) of 128 / RPT x 16 holds rows RPT tr .. and columns
// 8 tc .. +7 in registers, so a row's block is 16 neighbouring lanes (their maximum is four lane
// rotations) and a column's block is one thread's RPT rows and 128 / RPT threads, joined in LDS.  x is read once
// for both forms.  The transposed codes go through LDS so that each column's 128 codes leave as one line.
// The pass is bound by HBM: 2 or 4 bytes in and 1 or 2 out per element (8192x8192 bf16, both forms: 57 us, 4.8 TB/s,
// where a copy of 2 GiB reaches 4.9).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "sk_common.h"
#include "sk_fp8.h"

namespace sk {

namespace {

constexpr int kPitch = 136;   // LDS bytes between two columns' transposed codes: 34 banks

// Up to this many tiles have twice the threads each (4 rows a thread instead of 8), so that a SIMD has two waves where
// it would have one: 16x4096 3.4 -> 2.6 us, 1037x2050 both forms 7.3 -> 6.7, 2048x4096 both 11.2 -> 10.5; from
// 1024 tiles on (4096x4096 both, 16.8 against 16.9 us) there are enough waves without.
constexpr int64_t kFewTiles = 512;

// Byte of rows r .. of column c (r a multiple of RPT): 8-row pieces are moved by columns / 32, so that the lanes of a
// store (columns 8 apart, consecutive rows) meet each bank as often as their bytes need.
__device__ __forceinline__ int t_at(int c, int r) { return c * kPitch + ((r & ~7) ^ (32 * ((c >> 5) & 3))) + (r & 7); }

// 4 rows x 8 columns of codes (row i: w[i][0], w[i][1]) to 8 columns of 4 codes.
__device__ __forceinline__ void transpose4(const uint32_t (*w)[2], uint32_t (&o)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {      // columns 4 h .. +3
    const uint32_t a = w[0][h], b = w[1][h], c = w[2][h], d = w[3][h];
    // perm(hi, lo): selector bytes 0-3 pick from lo, 4-7 from hi
    const uint32_t ab0 = __builtin_amdgcn_perm(b, a, 0x05010400u), ab1 = __builtin_amdgcn_perm(b, a, 0x07030602u);
    const uint32_t cd0 = __builtin_amdgcn_perm(d, c, 0x05010400u), cd1 = __builtin_amdgcn_perm(d, c, 0x07030602u);
    o[4 * h] = __builtin_amdgcn_perm(cd0, ab0, 0x05040100u);
    o[4 * h + 1] = __builtin_amdgcn_perm(cd0, ab0, 0x07060302u);
    o[4 * h + 2] = __builtin_amdgcn_perm(cd1, ab1, 0x05040100u);
    o[4 * h + 3] = __builtin_amdgcn_perm(cd1, ab1, 0x07060302u);
  }
}

// TILE: one scale per 128 x 128.  PLAIN / TRANS: which forms are written (with SUMS: perhaps neither).  SUMS: also the
// column sums of the tile's rows, part[row block][column], in a fixed order (the first pass of a bias gradient).
template <class T, bool TILE, bool PLAIN, bool TRANS, bool SUMS, bool SHORT, int RPT>
__global__ __launch_bounds__(2048 / RPT) void sk_quantize_block(QuantArgs a) {
  static_assert(RPT == 8 || RPT == 4, "rows of a thread");
  constexpr int TR = 128 / RPT;         // threads of a column
  constexpr bool COLS = TRANS && !TILE;
  __shared__ __attribute__((aligned(16))) uint8_t codes_t[TRANS ? 128 * kPitch : 16];
  __shared__ __attribute__((aligned(16))) uint32_t tops[COLS ? TR : 1][128];
  constexpr bool LIFT = COLS && sizeof(T) == 4;   // columns of small scales are multiplied (see Coder<float>)
  __shared__ __attribute__((aligned(16))) float col_scale[LIFT ? 4 : COLS ? 3 : 1][128];
  __shared__ bool any_small;
  __shared__ __attribute__((aligned(16))) float col_sum[SUMS ? TR : 1][128];
  const int rb = blockIdx.x / a.kb, cb = blockIdx.x - rb * a.kb;
  const int t = threadIdx.x, tr = t >> 4, tc = t & 15;
  const int R = a.R, C = a.C;
  const int row0 = rb * 128 + RPT * tr, col0 = cb * 128 + 8 * tc;
  float x[RPT][8];
  {
    Raw8<T> raw[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) raw[i] = load_raw8<SHORT>((const T*)a.x + (int64_t)min(row0 + i, R - 1) * C, col0, C);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      settle8<SHORT>(raw[i], col0, C);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[i][k] = row0 + i < R ? raw_at(raw[i], k) : 0.0f;
    }
  }

  if constexpr (SUMS) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float s = x[0][k];
#pragma unroll
      for (int i = 1; i < RPT; ++i) s += x[i][k];
      col_sum[tr][8 * tc + k] = s;
    }
  }
  if constexpr (COLS) {
    if (LIFT && t == 0) any_small = false;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < RPT; ++i) m = max(m, f_bits(x[i][k]) & kAbs);
      tops[tr][8 * tc + k] = m;
    }
  }
  BlockScale tile;
  if constexpr (TILE) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < RPT; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) m = max(m, f_bits(x[i][k]) & kAbs);
    m = max16(m);
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    if ((t & 63) == 0) tops[0][t >> 6] = m;
    __syncthreads();
    m = tops[0][0];
#pragma unroll
    for (int w = 1; w < 32 / RPT; ++w) m = max(m, tops[0][w]);
    tile = Coder<T>::scale(m);
    if (t == 0) {
      if (PLAIN) a.scale[(int64_t)rb * a.kb + cb] = tile.s;
      if (TRANS) a.scale_t[(int64_t)cb * a.rb + rb] = tile.s;
    }
  } else if constexpr (COLS || SUMS) {
    __syncthreads();
    if (t < 128) {
      const int c = cb * 128 + t;
      if constexpr (COLS) {
        uint32_t m = tops[0][t];
#pragma unroll
        for (int i = 1; i < TR; ++i) m = max(m, tops[i][t]);
        BlockScale b = Coder<T>::scale(m);
        if (c < C) a.scale_t[(int64_t)rb * C + c] = b.s;
        if constexpr (LIFT) {
          if (Coder<T>::small(b)) any_small = true;
          col_scale[3][t] = Coder<T>::lift(b);
        }
        col_scale[0][t] = b.s;
        col_scale[1][t] = b.r;
        col_scale[2][t] = b.c;
      }
      if constexpr (SUMS) {
        float s = col_sum[0][t];
#pragma unroll
        for (int i = 1; i < TR; ++i) s += col_sum[i][t];
        if (c < C) a.part[(int64_t)rb * C + c] = s;
      }
    }
    if constexpr (COLS) __syncthreads();
  }

  // the rows' codes, eight bytes a lane: 16 lanes write a row's 128
  [[maybe_unused]] uint32_t w[RPT][2];
  if constexpr (PLAIN || TILE) {
    float own = 0.0f;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      BlockScale b;
      if constexpr (TILE) {
        b = tile;
      } else {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) m = max(m, f_bits(x[i][k]) & kAbs);
        b = Coder<T>::scale(max16(m));
        own = tc == i ? b.s : own;
      }
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = x[i][k];
      Coder<T>::nudge(v, b);
      w[i][0] = codes4(v[0], v[1], v[2], v[3], b.s);
      w[i][1] = codes4(v[4], v[5], v[6], v[7], b.s);
      // rows hold C rounded up to 16 codes, so a piece of eight is inside or outside as a whole
      if (PLAIN && row0 + i < R && col0 < a.pitch)
        *(u32x2*)(a.q + (int64_t)(row0 + i) * a.pitch + col0) = u32x2{w[i][0], w[i][1]};
    }
    if (!TILE && tc < RPT && row0 + tc < R) a.scale[(int64_t)cb * R + row0 + tc] = own;
  }

  if constexpr (TRANS) {
    uint32_t o[RPT / 4][8];    // rows 4 v .. +3 of each column
    if constexpr (TILE) {
#pragma unroll
      for (int v = 0; v < RPT / 4; ++v) transpose4(w + 4 * v, o[v]);
    } else {
      if constexpr (LIFT) {
        if (__builtin_expect(any_small, 0)) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int i = 0; i < RPT; ++i) x[i][k] *= col_scale[3][8 * tc + k];
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const BlockScale b{col_scale[0][8 * tc + k], col_scale[1][8 * tc + k], col_scale[2][8 * tc + k]};
        float v[RPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i) v[i] = x[i][k];
        if constexpr (LIFT) Coder<T>::nudge_lifted(v, b);
        else Coder<T>::nudge(v, b);
#pragma unroll
        for (int i = 0; i < RPT; i += 4) o[i / 4][k] = codes4(v[i], v[i + 1], v[i + 2], v[i + 3], b.s);
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint8_t* const to = codes_t + t_at(8 * tc + k, RPT * tr);
      if constexpr (RPT == 8) *(u32x2*)to = u32x2{o[0][k], o[RPT / 4 - 1][k]};
      else *(uint32_t*)to = o[0][k];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RPT / 2; ++i) {
      const int c = (t >> 3) + 256 / RPT * i, p = t & 7;     // column of the tile, 16 of its rows
      const uint8_t* from = codes_t + t_at(c, 16 * p);
      const u32x2 lo = *(const u32x2*)from, hi = *(const u32x2*)(from + 8);
      if (cb * 128 + c < C && rb * 128 + 16 * p < a.pitch_t)
        *(u32x4*)(a.qt + (int64_t)(cb * 128 + c) * a.pitch_t + rb * 128 + 16 * p) = u32x4{lo[0], lo[1], hi[0], hi[1]};
    }
  }
}

template <class T, bool TILE, bool SUMS, bool SHORT, int RPT>
hipError_t launch_form(const QuantArgs& a, hipStream_t s) {
  auto go = [&](auto kernel) { return launch(kernel, dim3((unsigned)a.kb * (unsigned)a.rb), 2048 / RPT, s, a); };
  if (a.q && a.qt) return go(sk_quantize_block<T, TILE, true, true, SUMS, SHORT, RPT>);
  if (a.q) return go(sk_quantize_block<T, TILE, true, false, SUMS, SHORT, RPT>);
  if (a.qt) return go(sk_quantize_block<T, TILE, false, true, SUMS, SHORT, RPT>);
  if constexpr (SUMS) return go(sk_quantize_block<T, TILE, false, false, SUMS, SHORT, RPT>);
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_quantize_block(const QuantArgs& a, bool f32, bool tile, hipStream_t s) {
  if (a.part && (f32 || tile)) return hipErrorInvalidValue;
  auto go = [&](auto elem, auto tiled, auto sums) {
    typedef decltype(elem) T;
    constexpr bool TILE = decltype(tiled)::value, SUMS = decltype(sums)::value;
    if (a.C < 8) return launch_form<T, TILE, SUMS, true, 8>(a, s);
    if ((int64_t)a.kb * a.rb <= kFewTiles) return launch_form<T, TILE, SUMS, false, 4>(a, s);
    return launch_form<T, TILE, SUMS, false, 8>(a, s);
  };
  const std::true_type yes;
  const std::false_type no;
  if (a.part) return go(uint16_t{}, no, yes);
  if (f32) return tile ? go(float{}, yes, no) : go(float{}, no, no);
  return tile ? go(uint16_t{}, yes, no) : go(uint16_t{}, no, no);
}

}  // namespace sk

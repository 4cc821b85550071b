// Products of few rows: C[m][n] = sum_k x[m][k] W[n][k] + bias[n], with one weight or, for rows sorted by expert, one
// for each expert.  The weight is 16-bit, or 4-bit codes with a 16-bit scale (and a zero point) for each group along K:
//
//   C[m][n] = sum_g s[g][n] ( sum_{k in g} (16 + q[n][k]) x[m][k] - (16 + z[g][n]) sum_{k in g} x[m][k] ) + bias[n]
//
// 16 + q is what four code bits become with one mask in a 16-bit float of exponent 4, exactly, so a pair of codes costs
// a shift and an and-or.  A group's inner sum is MFMAs' (16 rows of W by 16 of x, 32 of K), and so is the sum of x, with
// ones in place of W: its product with -(16 + z) is what the inner sum starts from (or is taken off it, where zero
// points differ).  The offset of 16 costs little precision: the terms are about five times the exact ones, in fp32.
//
// A workgroup takes 16 FN rows of W; its waves share out K in steps of 128 in turn, so that together they read whole
// stretches of a row, straight to registers, and their sums are added in order through LDS.

#include "sk_grouped.h"

namespace sk {

namespace {

constexpr int kStep = 128;   // of K, for a wave

// The matrix a[i][quarter of the wave] of registers transposed: register i of quarter q becomes register q of quarter i.
__device__ __forceinline__ void transpose4(v4u& a) {
  auto swap32 = [](uint32_t& x, uint32_t& y) {
    const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
    x = r[0];
    y = r[1];
  };
  auto swap16 = [](uint32_t& x, uint32_t& y) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, y, false, false);
    x = r[0];
    y = r[1];
  };
  uint32_t w[4] = {a[0], a[1], a[2], a[3]};
  swap32(w[0], w[2]);
  swap32(w[1], w[3]);
  swap16(w[0], w[1]);
  swap16(w[2], w[3]);
  a = v4u{w[0], w[1], w[2], w[3]};
}

// Eight codes as 16 + q in 16-bit floats, pairs (i, i + 4).
template <class T>
__device__ __forceinline__ v4u decode8(uint32_t d) {
  constexpr bool BF = std::is_same_v<T, Bf16>;
  constexpr uint32_t mask = BF ? 0x00780078u : 0x03c003c0u, base = BF ? 0x41804180u : 0x4c004c00u;
  constexpr int at = BF ? 3 : 6;         // where the code's bits go
  return v4u{(d << at & mask) | base, ((at >= 4 ? d << (at - 4) : d >> (4 - at)) & mask) | base,
             (d >> (8 - at) & mask) | base, (d >> (12 - at) & mask) | base};
}
// Eight elements in the same order.
__device__ __forceinline__ v4u pairs8(v4u x) {
  return v4u{__builtin_amdgcn_perm(x[2], x[0], 0x05040100u), __builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
             __builtin_amdgcn_perm(x[3], x[1], 0x05040100u), __builtin_amdgcn_perm(x[3], x[1], 0x07060302u)};
}

__device__ __forceinline__ v4u buffer16(const v4u& rsrc, uint32_t off) {
  return __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(rsrc_of(rsrc), (int)off, 0, 0));
}

// GROUP 0: 16-bit weights.  MT blocks of 16 rows of x, FN of 16 rows of W.
template <class T, int GROUP, bool ZERO, int FN, int MT, int NWK>
__global__ __launch_bounds__(64 * NWK) void sk_rows(RowsGemm g) {
  constexpr bool W4 = GROUP != 0;
  constexpr int WB = W4 ? kStep / 2 : kStep * 2;          // bytes of a row of W in a step
  constexpr int WL = W4 ? 1 : 4;                          // 16-byte loads of a lane, row block and step
  constexpr int NG = W4 ? kStep / GROUP : 1, PER = 4 / NG;   // groups of a step; MFMAs of a group
  __shared__ v4f red[NWK][FN * MT][64];
  const int lane = threadIdx.x & 63, wave = wave_id(), lr = lane & 15, lg = lane >> 4;
  const int n0 = blockIdx.x * 16 * FN;
  int e = 0, r0 = 0, r1 = g.R;
  bool zeros = false;
  if (g.offsets) {
    e = blockIdx.y;
    group_rows(g.offsets, e, g.E, g.R, &r0, &r1);
    r0 = __builtin_amdgcn_readfirstlane(r0);
    r1 = __builtin_amdgcn_readfirstlane(r1);
    if (e == g.E) {
      zeros = true;
      e = 0;
    }
  } else {
    r0 = min((int)blockIdx.y * 16 * MT, g.R);
    r1 = min(r0 + 16 * MT, g.R);
  }
  if (zeros) {
    for (int64_t r = r0 + wave; r < r1; r += NWK)
      for (int n = n0 + lane; n < min(n0 + 16 * FN, g.N); n += 64) g.C[r * g.N + n] = 0;
    return;
  }
  const uint32_t wrow = W4 ? (uint32_t)g.K / 2 : (uint32_t)g.K * 2, xrow = (uint32_t)g.K * 2;
  const int groups = W4 ? g.K / GROUP : 0;
  const v4u wr = rsrc_words(g.W + ((uint64_t)e * g.N + n0) * wrow, (uint32_t)min(16 * FN, g.N - n0) * wrow);
  const uint16_t* const scale = (const uint16_t*)g.scale + (uint64_t)e * groups * g.N;
  const uint8_t* const zero = ZERO ? g.zero + (uint64_t)e * groups * g.N : nullptr;
  const int steps = (g.K + kStep - 1) / kStep;

  for (int m0 = r0; m0 < r1; m0 += 16 * MT) {
    // the lane's row of x in each block, and its piece of W's rows
    const uint8_t* xp[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      int r = min(m0 + i * 16 + lr, r1 - 1);
      if (g.rows) r = min(max(g.rows[r], 0), g.x_rows - 1);
      xp[i] = g.x + (uint64_t)r * xrow;
    }
    v4f acc[FN][MT];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[j][i] = v4f{};

    for (int s = wave; s < steps; s += NWK) {
      const int k0 = s * kStep;
      v4u w[FN][WL], x[MT][4];
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int u = 0; u < WL; ++u) {
          const uint32_t at = (uint32_t)s * WB + (W4 ? 16 * lg : 64 * u + 16 * lg);
          w[j][u] = buffer16(wr, at < wrow ? (uint32_t)(j * 16 + lr) * wrow + at : kOob);
        }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int k = k0 + u * 32 + lg * 8;
          x[i][u] = k < g.K ? *(const v4u*)(xp[i] + (uint32_t)k * 2) : v4u{};
        }
      if constexpr (!W4) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[j][i] = T::mfma(w[j][u], x[i][u], acc[j][i]);
      } else {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int u = 0; u < 4; ++u) x[i][u] = pairs8(x[i][u]);
        const v4u ones{T::kOnes, T::kOnes, T::kOnes, T::kOnes};
        v4f sum[NG][MT];       // of x over a group, the same in all four
#pragma unroll
        for (int h = 0; h < NG; ++h)
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            sum[h][i] = v4f{};
#pragma unroll
            for (int u = 0; u < PER; ++u) sum[h][i] = T::mfma(ones, x[i][h * PER + u], sum[h][i]);
          }
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          transpose4(w[j][0]);
#pragma unroll
          for (int h = 0; h < NG; ++h) {
            v4u d[PER];
#pragma unroll
            for (int u = 0; u < PER; ++u) d[u] = decode8<T>(w[j][0][h * PER + u]);
            // scales of the lane's four rows of W (past N, or past the last group, any: nothing is made of them)
            const int64_t at = (int64_t)min(k0 / GROUP + h, groups - 1) * g.N;
            const int n = n0 + j * 16 + 4 * lg;
            float sc[4], z[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint16_t b = scale[at + min(n + c, g.N - 1)];
              sc[c] = T::lo(b);
              z[c] = ZERO ? (float)zero[at + min(n + c, g.N - 1)] : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              const float start = (ZERO ? -16.0f : -24.0f) * sum[h][i][0];
              v4f part{start, start, start, start};
#pragma unroll
              for (int u = 0; u < PER; ++u) part = T::mfma(d[u], x[i][h * PER + u], part);
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const float p = ZERO ? __builtin_fmaf(-z[c], sum[h][i][0], part[c]) : part[c];
                acc[j][i][c] = __builtin_fmaf(sc[c], p, acc[j][i][c]);
              }
            }
          }
        }
      }
    }
    // the waves' sums in order; block b is finished by wave b % NWK
    __syncthreads();
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int i = 0; i < MT; ++i) red[wave][j * MT + i][lane] = acc[j][i];
    __syncthreads();
    for (int b = wave; b < FN * MT; b += NWK) {
      v4f y = red[0][b][lane];
      for (int w = 1; w < NWK; ++w) y += red[w][b][lane];
      const int n = n0 + (b / MT) * 16 + 4 * lg, m = m0 + (b % MT) * 16 + lr;
      if (g.bias) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (n + c < g.N) y[c] += T::lo(g.bias[(uint64_t)e * g.N + n + c]);
      }
      if (m < r1 && n < g.N) store4<T>(g.C + (uint64_t)m * g.N + n, n, g.N, y[0], y[1], y[2], y[3]);
    }
  }
}

template <class T, int GROUP, bool ZERO>
hipError_t launch_rows_of(const RowsGemm& g, int cus, hipStream_t s) {
  constexpr int FN = 1, NWK = 8;
  const int groups = g.E + (g.tail ? 1 : 0);
  auto go = [&](auto mt) {
    constexpr int MT = decltype(mt)::value;
    const int64_t y = g.offsets ? groups : cdiv(g.R, 16 * MT);
    if (y > 65535) return hipErrorInvalidValue;
    return launch(sk_rows<T, GROUP, ZERO, FN, MT, NWK>, dim3((unsigned)cdiv(g.N, 16 * FN), (unsigned)y), 64 * NWK, s, g);
  };
  if (!g.offsets && g.R > 16) return go(std::integral_constant<int, 4>{});
  return go(std::integral_constant<int, 1>{});
}

template <class T, bool ZERO>
hipError_t by_group(const RowsGemm& g, int group, int cus, hipStream_t s) {
  if (group == 32) return launch_rows_of<T, 32, ZERO>(g, cus, s);
  if (group == 64) return launch_rows_of<T, 64, ZERO>(g, cus, s);
  return launch_rows_of<T, 128, ZERO>(g, cus, s);
}

}  // namespace

hipError_t launch_rows_w4(const RowsGemm& g, int group, bool f16, int cus, hipStream_t s) {
  if (f16) return g.zero ? by_group<Fp16, true>(g, group, cus, s) : by_group<Fp16, false>(g, group, cus, s);
  return g.zero ? by_group<Bf16, true>(g, group, cus, s) : by_group<Bf16, false>(g, group, cus, s);
}
hipError_t launch_rows_16(const RowsGemm& g, bool f16, int cus, hipStream_t s) {
  return f16 ? launch_rows_of<Fp16, 0, false>(g, cus, s) : launch_rows_of<Bf16, 0, false>(g, cus, s);
}

}  // namespace sk

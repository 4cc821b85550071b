// Products of few rows with 4-bit weights, one weight or, for rows sorted by expert, one for each expert: codes with a 16-bit scale
// (and a zero point) for each group along K,
//
//   C[m][n] = sum_g s[g][n] ( sum_{k in g} (16 + q[n][k]) x[m][k] - (16 + z[g][n]) sum_{k in g} x[m][k] ) + bias[n]
//
// 16 + q is what four code bits become with one mask in a 16-bit float of exponent 4, exactly, so a pair of codes costs
// a shift and an and-or.  A group's inner sum is MFMAs' (16 rows of W by 16 of x, 32 of K), and so is the sum of x, with
// -16 or -24 in place of W: what the inner sum starts from (other zero points are taken off it).  The offset of 16 costs little
// precision: the terms are about five times the exact ones, in fp32.  bf16 has fp32's range, so that 128 times 31 x would pass it for
// x above 2^116: there the float has exponent -8, all sums are 2^-12 of the formula's (128 x 31 < 2^12), and the output's sum is
// multiplied by 2^12.  (Powers of two: the same bits as without, but for sums below 2^-114, whose smallest step is 2^-137.)
//
// A workgroup takes 16 FN rows of W; its waves share out K in steps of 128 in turn, so that together they read whole
// stretches of a row, straight to registers and D steps ahead.  x lies in LDS, its elements in the order that the codes come in
// (KC of K at a time, where the rows are too many for all of it).  The waves' sums are added in order through LDS.

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

// Eight codes as 16 + q, by 2^-12 in bf16, in 16-bit floats, pairs (i, i + 4).  (`base` in a vector register and the mask in a scalar one: with two
// constants an and and an or would not be one instruction.)
template <class T>
struct Decode {
  static constexpr bool BF = std::is_same_v<T, Bf16>;
  static constexpr int at = BF ? 3 : 6;         // where the code's bits go
  uint32_t mask = BF ? 0x00780078u : 0x03c003c0u, base = BF ? 0x3b803b80u : 0x4c004c00u;
  __device__ __forceinline__ Decode() { asm volatile("" : "+s"(mask), "+v"(base)); }
  __device__ __forceinline__ v4u operator()(uint32_t d) const {
    return v4u{(d << at & mask) | base, ((at >= 4 ? d << (at - 4) : d >> (4 - at)) & mask) | base,
               (d >> (8 - at) & mask) | base, (d >> (12 - at) & mask) | base};
  }
};
// Eight elements in the same order.
__device__ __forceinline__ v4u pairs8(v4u x) {
  return v4u{__builtin_amdgcn_perm(x[2], x[0], 0x05040100u), __builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
             __builtin_amdgcn_perm(x[3], x[1], 0x05040100u), __builtin_amdgcn_perm(x[3], x[1], 0x07060302u)};
}

__device__ __forceinline__ v4u buffer16(const v4u& rsrc, uint32_t off) {
  return __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(rsrc_of(rsrc), (int)off, 0, 0));
}

// Scales or zero points of a lane's four rows of W, from a row of them at `base` of which there are n; those past the end, or of no
// step at all, are 0.
template <bool WIDE>
__device__ __forceinline__ v2u load_scales(const uint16_t* base, uint32_t n, uint32_t at) {
  const v4u r = rsrc_words(base, n * 2);
  if constexpr (WIDE) {
    return __builtin_bit_cast(v2u, __builtin_amdgcn_raw_buffer_load_b64(rsrc_of(r), (int)(at * 2), 0, 0));
  } else {
    uint32_t u[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) u[c] = __builtin_amdgcn_raw_buffer_load_b16(rsrc_of(r), (int)((at + c) * 2), 0, 0);
    return v2u{u[0] | u[1] << 16, u[2] | u[3] << 16};
  }
}
template <bool WIDE>
__device__ __forceinline__ uint32_t load_zeros(const uint8_t* base, uint32_t n, uint32_t at) {
  const v4u r = rsrc_words(base, n);
  if constexpr (WIDE) {
    return __builtin_amdgcn_raw_buffer_load_b32(rsrc_of(r), (int)at, 0, 0);
  } else {
    uint32_t u = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) u |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(rsrc_of(r), (int)(at + c), 0, 0) << (8 * c);
    return u;
  }
}

// What a wave holds of a step ahead of its use: codes, scales and zero points of 16 FN rows of W.
template <int FN, int NG>
struct Step {
  v4u code[FN];
  v2u scale[FN][NG];
  uint32_t zero[FN][NG];
};

// MT blocks of 16 rows of x, FN of 16 rows of W, NWK waves, D steps ahead.  WIDE: N is a multiple of 4 and scales are aligned to four.
template <class T, int GROUP, bool ZERO, bool WIDE, int FN, int MT, int NWK, int D>
__global__ __launch_bounds__(64 * NWK, MT == 1 ? 4 : 2) void sk_rows(RowsGemm g) {
  constexpr int NG = kStep / GROUP, PER = 4 / NG;      // groups of a step; MFMAs of a group
  constexpr int NT = 64 * NWK;
  extern __shared__ __attribute__((aligned(256))) uint8_t rows_smem[];
  const uint32_t smem = (uint32_t)(uintptr_t)(lds_u8*)rows_smem;
  const int lane = threadIdx.x & 63, wave = wave_id(), lr = lane & 15, lg = lane >> 4;
  // Each XCD (workgroups are dealt to them in turn) has neighbouring rows of W, whose scales lie in the same lines.
  const int x = blockIdx.x & 7, per = (int)gridDim.x >> 3, n0 = (x * per + min(x, (int)gridDim.x & 7) + ((int)blockIdx.x >> 3)) * 16 * FN;
  int e = 0, r0, r1;
  if (g.offsets) {
    e = blockIdx.y;
    group_rows(g.offsets, e, g.E, g.R, &r0, &r1);
    r0 = __builtin_amdgcn_readfirstlane(r0);
    r1 = __builtin_amdgcn_readfirstlane(r1);
    if (e == g.E) {       // rows behind the last expert's
      for (int64_t r = r0 + wave; r < r1; r += NWK)
        for (int n = n0 + lane; n < min(n0 + 16 * FN, g.N); n += 64) g.C[r * g.N + n] = 0;
      return;
    }
  } else {
    r0 = (int)min((int64_t)blockIdx.y * 16 * MT, (int64_t)g.R);
    r1 = min(r0 + 16 * MT, g.R);
  }
  const Decode<T> decode;
  const uint32_t wrow = (uint32_t)g.K / 2, xrow = (uint32_t)g.K * 2;
  const int groups = g.K / GROUP, steps = (g.K + kStep - 1) / kStep;
  const v4u wr = rsrc_words(g.W + ((uint64_t)e * g.N + n0) * wrow, (uint32_t)min(16 * FN, g.N - n0) * wrow);
  const uint16_t* const scale = (const uint16_t*)g.scale + (uint64_t)e * groups * g.N;
  const uint8_t* const zero = ZERO ? g.zero + (uint64_t)e * groups * g.N : nullptr;

  // A step's part of W (out of range, which costs no traffic, behind the last).
  auto load = [&](Step<FN, NG>& to, int s, int end) {
    const bool live = s < end;
    const uint32_t at = (uint32_t)s * (kStep / 2) + 16 * lg;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      to.code[j] = buffer16(wr, live && at < wrow ? (uint32_t)(j * 16 + lr) * wrow + at : kOob);
#pragma unroll
      for (int h = 0; h < NG; ++h) {
        const int gi = min(s * NG + h, groups - 1);       // (past the last group x is 0: any scale will do)
        const uint32_t n = live ? (uint32_t)(n0 + j * 16 + 4 * lg) : kOob / 4;
        to.scale[j][h] = load_scales<WIDE>(scale + (int64_t)gi * g.N, (uint32_t)g.N, n);
        if constexpr (ZERO) to.zero[j][h] = load_zeros<WIDE>(zero + (int64_t)gi * g.N, (uint32_t)g.N, n);
      }
    }
  };
  // Where eight elements of x (chunk c of a row) lie in its row: the order of a step's 16 chunks follows that of the codes (a lane
  // has 32 of a row, which for groups of 128 stay where they are and else are exchanged between the lanes), and rows are
  // permuted by their number, so that 16 lanes which read a chunk of 16 rows meet every bank once.
  auto x_at = [&](int kc, int m, int c) {
    const int in = GROUP == 128 ? (c & 3) << 2 | (c >> 2 & 3) : c & 15;
    return (uint32_t)m * (uint32_t)kc * 2u + (uint32_t)((c & ~15) | (in ^ (m & 15))) * 16u;
  };

  for (int m0 = r0; m0 < r1; m0 += 16 * MT) {
    const int rows = min(16 * MT, r1 - m0);
    // of K, that LDS holds of these rows: all of it, or whole turns of the waves
    const int fit = g.lds / (2 * rows);
    const int kc = steps * kStep <= fit ? steps * kStep : fit / (kStep * NWK) * (kStep * NWK);
    v4f acc[FN][MT];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[j][i] = v4f{};

    for (int kb = 0; kb < g.K; kb += kc) {
      const int first = kb / kStep, end = min(steps, first + kc / kStep);
      Step<FN, NG> ahead[D];
#pragma unroll
      for (int d = 0; d < D; ++d) load(ahead[d], first + wave + d * NWK, end);
      __syncthreads();       // the last part of x, or the last sums, have been read
      // several rows' loads at a time (one by one, each waited for, 8 rows of 4096 took 10 us more in all)
      const int chunks = (end - first) * 16;
      auto stage = [&](auto rows_at_once, int mb) {
        constexpr int Q = decltype(rows_at_once)::value;
        const uint8_t* from[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          int r = m0 + min(mb + q, rows - 1);
          if (g.rows) r = min(__builtin_amdgcn_readfirstlane(max(g.rows[r], 0)), g.x_rows - 1);
          from[q] = g.x + (uint64_t)r * xrow;
        }
        for (int c = threadIdx.x; c < chunks; c += NT) {
          const uint32_t k = (uint32_t)(kb + c * 8);
          v4u v[Q];
#pragma unroll
          for (int q = 0; q < Q; ++q) v[q] = k < (uint32_t)g.K ? *(const v4u*)(from[q] + k * 2) : v4u{};
#pragma unroll
          for (int q = 0; q < Q; ++q)
            if (mb + q < rows) *(__attribute__((address_space(3))) v4u*)(uintptr_t)(smem + x_at(kc, mb + q, c)) = pairs8(v[q]);
        }
      };
      int mb = 0;
      if constexpr (MT == 1)
        for (; mb + 4 < rows; mb += 8) stage(std::integral_constant<int, 8>{}, mb);
      for (; mb + 1 < rows; mb += 4) stage(std::integral_constant<int, 4>{}, mb);
      if (mb < rows) stage(std::integral_constant<int, 1>{}, mb);
      __syncthreads();
      for (int s0 = first + wave; s0 < end; s0 += NWK * D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
          const int s = s0 + d * NWK;
          if (s < end) {
            v4u x[MT][4];
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const int m = i * 16 + lr;
                // (chunk 4 u + lg of the stored order)
                const uint32_t at = (uint32_t)(m < rows ? m : 0) * (uint32_t)kc * 2u +
                                    (uint32_t)((s - first) * 16 + ((4 * u + lg) ^ (m < rows ? m & 15 : 0))) * 16u;
                x[i][u] = *(const __attribute__((address_space(3))) v4u*)(uintptr_t)(smem + at);
              }
            // -16 times x's sum over a group (-24 times without zero points; by 2^-12 in bf16), the same in all four: what its
            // products start from
            constexpr uint32_t by = ZERO ? T::kMinus16 : T::kMinus24;
            const v4u minus{by, by, by, by};
            v4f sum[NG][MT];
#pragma unroll
            for (int h = 0; h < NG; ++h)
#pragma unroll
              for (int i = 0; i < MT; ++i) {
                sum[h][i] = v4f{};
#pragma unroll
                for (int u = 0; u < PER; ++u) sum[h][i] = T::mfma(minus, x[i][h * PER + u], sum[h][i]);
              }
            float less[NG][MT];     // -x's sum (by 2^-12 in bf16)
#pragma unroll
            for (int h = 0; h < NG; ++h)
#pragma unroll
              for (int i = 0; i < MT; ++i) less[h][i] = sum[h][i][0] * 0.0625f;
#pragma unroll
            for (int j = 0; j < FN; ++j) {
              v4u code = ahead[d].code[j];
              if constexpr (GROUP != 128) transpose4(code);
#pragma unroll
              for (int h = 0; h < NG; ++h) {
                v4u q[PER];
#pragma unroll
                for (int u = 0; u < PER; ++u) q[u] = decode(code[h * PER + u]);
                const v2u sc = ahead[d].scale[j][h];
                const float f[4] = {T::lo(sc[0]), T::hi(sc[0]), T::lo(sc[1]), T::hi(sc[1])};
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                  v4f part = sum[h][i];
#pragma unroll
                  for (int u = 0; u < PER; ++u) part = T::mfma(q[u], x[i][h * PER + u], part);
#pragma unroll
                  for (int c = 0; c < 4; ++c) {
                    float y = part[c];
                    if constexpr (ZERO) y = __builtin_fmaf((float)(ahead[d].zero[j][h] >> (8 * c) & 255u), less[h][i], y);
                    acc[j][i][c] = __builtin_fmaf(f[c], y, acc[j][i][c]);
                  }
                }
              }
            }
          }
          load(ahead[d], s + NWK * D, end);
        }
      }
    }
    // the waves' sums in order; block b is finished by wave b % NWK
    auto red = [&](int w, int b) { return (__attribute__((address_space(3))) v4f*)(uintptr_t)(smem + (uint32_t)((w * FN * MT + b) * 64 + lane) * 16u); };
    __syncthreads();
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int i = 0; i < MT; ++i) *red(wave, j * MT + i) = acc[j][i];
    __syncthreads();
    for (int b = wave; b < FN * MT; b += NWK) {
      v4f y = *red(0, b);
#pragma unroll
      for (int w = 1; w < NWK; ++w) y += *red(w, b);
      if constexpr (Decode<T>::BF) y *= 0x1p12f;
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

template <class T, int GROUP, bool ZERO, bool WIDE, int FN, int MT, int NWK>
hipError_t launch_rows_as(RowsGemm g, hipStream_t s) {
  constexpr int D = MT > 1 || GROUP == 32 ? 1 : 2;
  const int groups = g.offsets ? g.E + (g.tail ? 1 : 0) : 1;
  const int64_t y = g.offsets ? groups : cdiv(g.R, 16 * MT);
  if (y > 65535) return hipErrorInvalidValue;
  // LDS for x: 16 waves to a unit, or 8 with many rows, and no more than all rows take
  constexpr int most = MT > 1 || NWK == 16 ? 128 * 1024 : NWK == 8 ? 64 * 1024 : 40 * 1024, least = NWK * FN * MT * 1024;
  static_assert(most / (2 * 16 * MT) >= kStep * NWK && least <= most, "a turn of the waves, and their sums");
  const int64_t all = 2 * (int64_t)(g.R < 16 * MT ? g.R : 16 * MT) * cdiv(g.K, kStep) * kStep;
  g.lds = all < least ? least : all > most ? most : (int)all;
  void* args[] = {&g};
  const hipError_t r = hipLaunchKernel((const void*)sk_rows<T, GROUP, ZERO, WIDE, FN, MT, NWK, D>,
                                       dim3((unsigned)cdiv(g.N, 16 * FN), (unsigned)y), dim3(64 * NWK), args, (size_t)g.lds, s);
  if (r != hipSuccess) (void)hipGetLastError();
  return r;
}

template <class T, int GROUP, bool ZERO>
hipError_t launch_rows_of(const RowsGemm& g, int cus, hipStream_t s) {
  const bool wide = g.N % 4 == 0 && ((uintptr_t)g.scale & 7) == 0 && ((uintptr_t)g.zero & 3) == 0;
  const int64_t per = g.offsets ? cdiv(g.R, g.E) : g.R;       // rows of a weight, about
  constexpr int MORE = GROUP == 32 ? 1 : 2;     // (the scales of 32 rows of groups of 32 do not fit the registers)
  if (g.offsets && per <= 8) {
    // Four waves to a workgroup: an expert's few rows are soon done, and several workgroups to a unit share what begins and ends
    // them (16 tokens x 2 of 8, 4096 x 4096, groups of 64 with zero points: 25.5 us against 28.1 with 8 waves and 40.1 with 16; here
    // and below calls among others, with weights from memory).
    if (!wide) return launch_rows_as<T, GROUP, ZERO, false, 1, 1, 4>(g, s);
    return launch_rows_as<T, GROUP, ZERO, true, MORE, 1, 4>(g, s);
  }
  if (!g.offsets && per <= 4) {
    // 1x8192x8192 11.0 us against 12.4 with 4 waves and 12.2 with 16
    if (!wide) return launch_rows_as<T, GROUP, ZERO, false, 1, 1, 8>(g, s);
    // 32 rows of W to a workgroup where half as many still fill the device (16384x8192 19.2 us against 22.7 with 16, 8192x8192 11.0 / 11.2,
    // 4096x4096 6.1 / 5.1)
    if (MORE > 1 && cdiv(g.N, 32) >= cus) return launch_rows_as<T, GROUP, ZERO, true, MORE, 1, 8>(g, s);
    return launch_rows_as<T, GROUP, ZERO, true, 1, 1, 8>(g, s);
  }
  if (!g.offsets && per <= 32) {
    // Every workgroup reads all of x: more waves to it (16x8192x8192 18.3 us against 22.1 with 8; 5 rows 13.1 / 13.4, but 32 rows 31.9 /
    // 28.7).  Up to 32 rows as two workgroups of 16 (32x8192x8192 31.9 us against 42.0 with 32 at a time; 64 rows 59.6 / 42.0).
    if (!wide) return launch_rows_as<T, GROUP, ZERO, false, 1, 1, 16>(g, s);
    return launch_rows_as<T, GROUP, ZERO, true, MORE, 1, 16>(g, s);
  }
  // 32 rows of x at a time; with more, the weight's second reading comes from the caches
  constexpr int MOST = GROUP == 32 ? 2 : 4;
  return wide ? launch_rows_as<T, GROUP, ZERO, true, MOST, 2, 8>(g, s) : launch_rows_as<T, GROUP, ZERO, false, 2, 2, 8>(g, s);
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
}  // namespace sk

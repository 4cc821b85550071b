// Products grouped by expert, for rows that lie sorted by expert (expert e has rows offsets[e] .. offsets[e + 1]):
//
//   forward   C[r][n]  = sum_k A[rows[r]][k] B[e][n][k] + bias[e][n]      (rows: optional, a gather)
//   dA        dA[r][k] = sum_n dC[r][n] B[e][n][k]
//   dB        dB[e][n][k] = sum_r dC[r][n] A[rows[r]][k],   dbias[e][n] = sum_r dC[r][n]
//
// The group sizes are known to the device alone.  The launch has a workgroup for the most tiles that R rows in E groups
// can make; each finds its tile from the offsets, and those past the last tile leave at once.  Rows behind
// the last group are a group of their own whose tiles are zeros (where the caller wants them written).
//
// One kernel for the three: an operand lies either with the dimension summed over contiguous (A, B forward, dC in
// dA) or with it as rows (B in dA, dC and A in dB).  Both kinds go straight from memory into LDS, 16 bytes a lane;
// the second kind is turned as it is read (ds_read_b64_tr_b16: of 16 lanes that read 4 rows of 16 elements, lane i
// gets column i), so nothing is transposed in memory.
#pragma once

#include "sk_fp8.h"
#include "sk_kernel.h"

namespace sk {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;
typedef unsigned v2u_any __attribute__((ext_vector_type(2), aligned(2)));

// The two element types: the matrix instruction, and rounding.
struct Bf16 {
  static __device__ __forceinline__ v4f mfma(v4u b, v4u a, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, b), __builtin_bit_cast(v8bf, a), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) { return pack_bf16(a, b); }
  static __device__ __forceinline__ float lo(uint32_t w) { return bf16_lo(w); }
  static __device__ __forceinline__ float hi(uint32_t w) { return bf16_hi(w); }
  static constexpr uint32_t kOnes = 0x3f803f80u;
};
struct Fp16 {
  static __device__ __forceinline__ v4f mfma(v4u b, v4u a, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, b), __builtin_bit_cast(v8h, a), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, (h2{(_Float16)a, (_Float16)b}));
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return (float)__builtin_bit_cast(_Float16, (uint16_t)w); }
  static __device__ __forceinline__ float hi(uint32_t w) { return (float)__builtin_bit_cast(_Float16, (uint16_t)(w >> 16)); }
  static constexpr uint32_t kOnes = 0x3c003c00u;
};

enum GroupedKind { kForward = 0, kGradA = 1, kGradB = 2 };

// Tile BM x BN of the output on WM x WN waves, k-steps of 64 of the dimension summed over, STAGES of them in LDS.
template <class T_, int KIND_, int BM_, int BN_, int WM_, int WN_, int STAGES_>
struct GroupedCfg {
  using T = T_;
  static constexpr int KIND = KIND_, BM = BM_, BN = BN_, WM = WM_, WN = WN_, STAGES = STAGES_;
  static constexpr int NW = WM * WN, NT = 64 * NW;
  static constexpr int WTM = BM / WM, WTN = BN / WN, FM = WTM / 16, FN = WTN / 16;
  static constexpr bool PT = KIND == kGradB, QT = KIND != kForward;   // operands to be turned
  static constexpr int P_BYTES = BM * 128, Q_BYTES = BN * 128, STAGE = P_BYTES + Q_BYTES;
  static constexpr int P_PT = BM / 8 / NW, Q_PT = BN / 8 / NW, D = P_PT + Q_PT;   // direct loads of a wave and k-step
  static constexpr int LDS = STAGES * STAGE;
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "whole loads for each wave");
  static_assert(LDS <= 160 * 1024, "LDS");
};

// How an operand of BX rows or columns lies in LDS and is loaded by NW waves.
//
// Not turned: 128 bytes of a row; the 16-byte chunks of row r are permuted by (r >> 1) & 7, so that 16 lanes that
// read a chunk of 16 rows meet every bank once.  A load of 64 lanes is 8 rows.
// Turned: a k-step's 64 rows of BX elements each; pairs of chunks are permuted by the row so that the 4 rows
// that 16 lanes read, and those of the next 16 lanes (8 rows on), lie in different banks.
template <int BX, int NW, bool TURN>
struct Operand {
  static constexpr int ROW = TURN ? BX * 2 : 128;                  // bytes of a row in LDS
  static constexpr int RPU = 1024 / ROW;                           // rows of a wave's load
  static constexpr int PER = BX / 8 / NW;                          // loads of a wave and k-step
  static_assert(!TURN || (BX >= 64 && BX <= 256), "the permutation below");

  // The permutation of a turned operand's row, in 16-byte chunks.
  static __device__ __forceinline__ int swizzle(int row) {
    if constexpr (BX == 64) return 2 * (((row >> 1) & 1) | ((row >> 3) & 1) << 1);
    else return 2 * ((row & 3) | ((row >> 3) & 1) << 2);
  }
  // Load i of wave w: the lane's row, and its chunk of that row.
  static __device__ __forceinline__ int row_of(int w, int i, int lane) { return (w + i * NW) * RPU + lane / (64 / RPU); }
  static __device__ __forceinline__ int chunk_of(int w, int i, int lane) {
    const int r = row_of(w, i, lane);
    if constexpr (!TURN) return (lane & 7) ^ ((r >> 1) & 7);
    else return (lane % (ROW / 16)) ^ swizzle(r);
  }
  // The lane's first address of its part of block 0 (16 rows or columns from `first`) in the stage at `base`.
  static __device__ __forceinline__ uint32_t read_base(uint32_t base, int first, int lane) {
    const int lr = lane & 15, lg = lane >> 4;
    if constexpr (!TURN) {
      return base + (uint32_t)((first + lr) * 128 + ((lg ^ ((lr >> 1) & 7)) * 16));
    } else {
      const int r = lg * 8 + (lr >> 2);
      return base + (uint32_t)(r * ROW + (((first / 8) ^ swizzle(r)) | ((lr >> 1) & 1)) * 16 + 8 * (lr & 1));
    }
  }
  // Block b's elements of half h (32 of the dimension summed over) from there.
  template <int H>
  static __device__ __forceinline__ v4u read(uint32_t at, int b) {
    if constexpr (!TURN) {
      return *(const __attribute__((address_space(3))) v4u*)(uintptr_t)((H ? at ^ 64u : at) + (uint32_t)b * 2048u);
    } else {
      const uint32_t a = (at ^ (uint32_t)(b * 32)) + H * 32 * ROW;
      const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(uintptr_t)a);
      const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(uintptr_t)(a + 4 * ROW));
      const v2u u = __builtin_bit_cast(v2u, x), w = __builtin_bit_cast(v2u, y);
      return v4u{u[0], u[1], w[0], w[1]};
    }
  }
};

// Rows [start, end) of group g, whatever the offsets hold.
__device__ __forceinline__ void group_rows(const int* offsets, int g, int E, int R, int* start, int* end) {
  *start = min(max(offsets[g], 0), R);
  *end = g < E ? min(max(offsets[g + 1], *start), R) : R;
}

struct GroupTile {
  int e;           // expert; E for the rows behind the last one's
  int row0, rows;  // the tile's rows
  int tn;          // its column of tiles
};

// The tile of workgroup t (false: none).  Groups in order, each in bands of BAND tile rows by all its columns, and the
// list of tiles cut into eight runs, one for each XCD (workgroups are dealt to them in turn), whose L2 then
// holds an expert's weights for several workgroups.
template <int BM, int BAND>
__device__ __forceinline__ bool find_tile(const int* offsets, int E, int R, int tiles_n, bool tail, int t, GroupTile* out) {
  const int lane = threadIdx.x & 63, G = E + (tail ? 1 : 0);
  auto tiles_of = [&](int g) {
    int a = 0, b = 0;
    if (g < G) group_rows(offsets, g, E, R, &a, &b);
    return (b - a + BM - 1) / BM;
  };
  auto scan = [&](int x) {       // inclusive, over the wave
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int y = __shfl_up(x, d);
      x += lane >= d ? y : 0;
    }
    return x;
  };
  const int first = scan(tiles_of(lane));
  int total = __builtin_amdgcn_readlane(first, 63);
  for (int g = 64; g < G; g += 64) {
    int x = tiles_of(g + lane);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) x += __shfl_xor(x, d);
    total += __builtin_amdgcn_readfirstlane(x);
  }
  const int64_t T = min((int64_t)total * tiles_n, (int64_t)gridDim.x);
  if (t >= T) return false;
  const int x = t & 7, per = (int)(T >> 3), rest = (int)(T & 7);
  const int i = x * per + min(x, rest) + (t >> 3);
  const int im = i / tiles_n;         // the tile row that the plain order would give: its group
  int base = 0, s = first;
  int g0 = 0;
  while (true) {
    const uint64_t before = __ballot(base + s <= im);
    if (~before || g0 + 64 >= G) {
      const int e = before == ~0ull ? 63 : __builtin_ctzll(~before);
      out->e = g0 + e;
      base += e ? __builtin_amdgcn_readlane(s, e - 1) : 0;
      break;
    }
    base += __builtin_amdgcn_readlane(s, 63);
    g0 += 64;
    s = scan(tiles_of(g0 + lane));
  }
  out->e = __builtin_amdgcn_readfirstlane(out->e);
  base = __builtin_amdgcn_readfirstlane(base);
  int a, b;
  group_rows(offsets, out->e, E, R, &a, &b);
  const int tm_e = (b - a + BM - 1) / BM;
  const int in = i - base * tiles_n, band = in / (BAND * tiles_n), at = in - band * BAND * tiles_n;
  const int rows = max(1, min(BAND, tm_e - band * BAND));
  const int tn = at / rows, tm = band * BAND + (at - tn * rows);
  out->row0 = __builtin_amdgcn_readfirstlane(a + tm * BM);
  out->rows = __builtin_amdgcn_readfirstlane(max(0, min(BM, b - a - tm * BM)));
  out->tn = __builtin_amdgcn_readfirstlane(tn);
  return out->rows > 0 && tn < tiles_n;
}

// Four outputs of a row from column n on, of which those below N are stored.
template <class T>
__device__ __forceinline__ void store4(uint16_t* p, int n, int N, float a, float b, float c, float d) {
  const v2u w{T::pack(a, b), T::pack(c, d)};
  if (n + 4 <= N) {
    *(v2u_any*)p = w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) p[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
  }
}

// P is the operand of the output's rows, Q that of its columns.
template <class C>
__device__ __forceinline__ void grouped_tile(const GroupedGemm& g, lds_u8* const smem) {
  using T = typename C::T;
  using OpP = Operand<C::BM, C::NW, C::PT>;
  using OpQ = Operand<C::BN, C::NW, C::QT>;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int wm = wave / C::WN, wn = wave % C::WN, lr = lane & 15, lg = lane >> 4;
  const uint32_t ring = (uint32_t)(uintptr_t)smem;

  // ---- what this workgroup computes
  int e, row0 = 0, rows = 0, m0 = 0, n0, steps;
  bool zeros = false;
  if constexpr (C::KIND == kGradB) {
    // expert e's [N][K], tile rows of N by tile columns of K, each XCD a run of tiles
    const int per_e = g.tiles_m * g.tiles_n, total = g.E * per_e, x = blockIdx.x & 7;
    const int i = x * (total >> 3) + min(x, total & 7) + (int)(blockIdx.x >> 3);
    e = i / per_e;
    const int at = i - e * per_e, tn = at / g.tiles_m;
    m0 = (at - tn * g.tiles_m) * C::BM;
    n0 = tn * C::BN;
    int end;
    group_rows(g.offsets, e, g.E, g.R, &row0, &end);
    row0 = __builtin_amdgcn_readfirstlane(row0);
    rows = __builtin_amdgcn_readfirstlane(end) - row0;
    steps = (rows + 63) / 64;
  } else {
    GroupTile t;
    if (!find_tile<C::BM, C::BM >= 256 ? 4 : 8>(g.offsets, g.E, g.R, g.tiles_n, g.tail, (int)blockIdx.x, &t)) return;
    e = t.e;
    row0 = t.row0;
    rows = t.rows;
    n0 = t.tn * C::BN;
    zeros = e >= g.E;
    steps = zeros ? 0 : (g.S + 63) / 64;
  }

  // ---- where the operands' loads come from
  uint32_t pvoff[C::P_PT], qvoff[C::Q_PT];
  v4u pr, qr;
  const uint32_t pp = (uint32_t)g.p_pitch, qp = (uint32_t)g.q_pitch;
  const uint64_t e_off = zeros ? 0 : (uint64_t)e;
  if constexpr (!C::PT) {
    if (g.rows && C::KIND == kForward) {
#pragma unroll
      for (int i = 0; i < C::P_PT; ++i) {
        const int r = min(OpP::row_of(wave, i, lane), rows - 1);
        const int t = zeros ? 0 : min(max(g.rows[row0 + r], 0), g.p_rows - 1);
        pvoff[i] = (uint32_t)t * pp + OpP::chunk_of(wave, i, lane) * 16;
      }
      pr = rsrc_words(g.P, (uint32_t)g.p_rows * pp);
    } else {
#pragma unroll
      for (int i = 0; i < C::P_PT; ++i)
        pvoff[i] = (uint32_t)OpP::row_of(wave, i, lane) * pp + OpP::chunk_of(wave, i, lane) * 16;
      pr = rsrc_words(g.P + (uint64_t)row0 * pp, (uint32_t)rows * pp);
    }
  } else {
#pragma unroll
    for (int i = 0; i < C::P_PT; ++i)
      pvoff[i] = (uint32_t)OpP::row_of(wave, i, lane) * pp + OpP::chunk_of(wave, i, lane) * 16;
  }
  if constexpr (!C::QT) {
#pragma unroll
    for (int i = 0; i < C::Q_PT; ++i)
      qvoff[i] = (uint32_t)OpQ::row_of(wave, i, lane) * qp + OpQ::chunk_of(wave, i, lane) * 16;
    qr = rsrc_words(g.Q + (e_off * g.Nout + n0) * qp, (uint32_t)min(C::BN, g.Nout - n0) * qp);
  } else {
#pragma unroll
    for (int i = 0; i < C::Q_PT; ++i)
      qvoff[i] = (uint32_t)OpQ::row_of(wave, i, lane) * qp + OpQ::chunk_of(wave, i, lane) * 16;
  }
  const bool gather_q = C::KIND == kGradB && g.rows;
  // Rows of the k-step at s of a turned operand: `have` rows from `base` on.
  auto turned = [&](const uint8_t* base, uint32_t pitch, int col0, int64_t have, int s) {
    const int64_t left = min(max(have - (int64_t)s * 64, (int64_t)0), (int64_t)64);
    const uint32_t bytes = left > 0 ? (uint32_t)left * pitch - (uint32_t)col0 * 2 : 0u;
    return rsrc_words(base + (uint64_t)s * 64 * pitch + (uint32_t)col0 * 2, bytes);
  };

  // The direct loads of k-step s, one at a time; past the last one every lane is out of range (zeros, no traffic).
  v4u ps, qs;       // the k-step's resources of turned operands
  auto aim = [&](int s) {
    if constexpr (C::PT) ps = turned(g.P + (uint64_t)row0 * pp, pp, m0, rows, s);
    if constexpr (C::QT) {
      if constexpr (C::KIND == kGradB) {
        if (gather_q) qs = rsrc_words(g.Q + n0 * 2, (uint32_t)g.q_rows * qp - (uint32_t)n0 * 2);
        else qs = turned(g.Q + (uint64_t)row0 * qp, qp, n0, rows, s);
      } else {
        qs = turned(g.Q + e_off * g.S * qp, qp, n0, g.S, s);
      }
    }
  };
  auto load = [&](int s, uint32_t stage, auto lc) {
    constexpr int l = decltype(lc)::value;
    const bool live = s < steps;
    const uint32_t kb = (uint32_t)s * 128u;       // of operands that are not turned
    if constexpr (l < C::P_PT) {
      const uint32_t at = stage + (uint32_t)(wave + l * C::NW) * 1024u;
      if constexpr (!C::PT) {
        const bool in = live && kb + OpP::chunk_of(wave, l, lane) * 16 < (uint32_t)g.S * 2u;
        dma_load16(pr, in ? pvoff[l] : kOob, live ? kb : 0u, at);
      } else {
        dma_load16(ps, live ? pvoff[l] : kOob, 0u, at);
      }
    } else {
      constexpr int i = l - C::P_PT;
      const uint32_t at = stage + C::P_BYTES + (uint32_t)(wave + i * C::NW) * 1024u;
      if constexpr (!C::QT) {
        const bool in = live && kb + OpQ::chunk_of(wave, i, lane) * 16 < (uint32_t)g.S * 2u;
        dma_load16(qr, in ? qvoff[i] : kOob, live ? kb : 0u, at);
      } else if (C::KIND == kGradB && gather_q) {
        const int r = s * 64 + OpQ::row_of(wave, i, lane);
        uint32_t v = kOob;
        if (r < rows) {
          const int t = min(max(g.rows[row0 + r], 0), g.q_rows - 1);
          v = (uint32_t)t * qp + OpQ::chunk_of(wave, i, lane) * 16;
        }
        dma_load16(qs, v, 0u, at);
      } else {
        dma_load16(qs, live ? qvoff[i] : kOob, 0u, at);
      }
    }
  };

  // ---- the k-steps
  v4f acc[C::FM][C::FN];
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) acc[i][j] = v4f{};
  constexpr bool SUMS = C::KIND == kGradB;
  v4f sums[SUMS ? C::FM : 1];
#pragma unroll
  for (int i = 0; i < (SUMS ? C::FM : 1); ++i) sums[i] = v4f{};
  const bool with_sums = SUMS && g.dbias && n0 == 0 && wn == 0;

  v4u p[2][C::FM], q[2][C::FN];
  uint32_t lp, lq;
  auto aim_reads = [&](int slot) {
    lp = OpP::read_base(ring + (uint32_t)slot * C::STAGE, wm * C::WTM, lane);
    lq = OpQ::read_base(ring + (uint32_t)slot * C::STAGE + C::P_BYTES, wn * C::WTN, lane);
  };
  // Read n of the FM + FN of a half, in the order in which the products need them.
  auto read = [&](auto hc, auto nc) {
    constexpr int h = decltype(hc)::value, n = decltype(nc)::value;
    if constexpr (n == 0) q[h][0] = OpQ::template read<h>(lq, 0);
    else if constexpr (n <= C::FM) p[h][n - 1] = OpP::template read<h>(lp, n - 1);
    else q[h][n - C::FM] = OpQ::template read<h>(lq, n - C::FM);
  };
  constexpr int NS = C::FM * C::FN, NR = C::FM + C::FN;

  if (steps > 0) {
    static_for<C::STAGES>([&](auto sc) {
      constexpr int s = decltype(sc)::value;
      aim(s);
      static_for<C::D>([&](auto l) { load(s, ring + s * C::STAGE, l); });
    });
    wait_vmcnt_n<C::D*(C::STAGES - 1)>();
    lds_barrier();
    aim_reads(0);
    static_for<NR>([&](auto n) { read(std::integral_constant<int, 0>{}, n); });
    int slot = 0;
    for (int s = 0; s < steps; ++s) {
      // first half: its products, and the second half's reads beside them
      static_for<NS>([&](auto nc) {
        constexpr int n = decltype(nc)::value, i = n % C::FM, j = n / C::FM;
        acc[i][j] = T::mfma(q[0][j], p[0][i], acc[i][j]);
        constexpr int R0 = n * NR / NS, R1 = (n + 1) * NR / NS;
        static_for<R1 - R0>([&](auto k) {
          read(std::integral_constant<int, 1>{}, std::integral_constant<int, R0 + decltype(k)::value>{});
        });
        __builtin_amdgcn_sched_barrier(0);
      });
      if constexpr (SUMS)
        if (with_sums) {
#pragma unroll
          for (int i = 0; i < C::FM; ++i) {
            const v4u ones{T::kOnes, T::kOnes, T::kOnes, T::kOnes};
            sums[i] = T::mfma(ones, p[0][i], sums[i]);
            sums[i] = T::mfma(ones, p[1][i], sums[i]);
          }
        }
      // the next k-step has arrived and this one has been read: its place is free
      const uint32_t freed = ring + (uint32_t)slot * C::STAGE;
      slot = slot + 1 == C::STAGES ? 0 : slot + 1;
      wait_vmcnt_n<C::D*(C::STAGES - 2)>();
      lds_barrier();
      aim_reads(slot);
      aim(s + C::STAGES);
      static_for<NS>([&](auto nc) {
        constexpr int n = decltype(nc)::value, i = n % C::FM, j = n / C::FM;
        acc[i][j] = T::mfma(q[1][j], p[1][i], acc[i][j]);
        constexpr int R0 = n * NR / NS, R1 = (n + 1) * NR / NS;
        static_for<R1 - R0>([&](auto k) {
          read(std::integral_constant<int, 0>{}, std::integral_constant<int, R0 + decltype(k)::value>{});
        });
        constexpr int L0 = n * C::D / NS, L1 = (n + 1) * C::D / NS;
        static_for<L1 - L0>([&](auto k) {
          load(s + C::STAGES, freed, std::integral_constant<int, L0 + decltype(k)::value>{});
        });
        __builtin_amdgcn_sched_barrier(0);
      });
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }

  // ---- outputs: the lane has row lr and columns 4 lg .. + 3 of each 16 x 16 block
  const uint16_t* const bias = C::KIND == kForward && g.bias && !zeros ? g.bias + (uint64_t)e * g.Nout : nullptr;
  uint16_t* const out = C::KIND == kGradB ? g.C + (uint64_t)e * g.Mout * g.Nout : g.C + (uint64_t)row0 * g.Nout;
  const int mrows = C::KIND == kGradB ? min(C::BM, g.Mout - m0) : rows;
#pragma unroll
  for (int j = 0; j < C::FN; ++j) {
    const int n = n0 + wn * C::WTN + j * 16 + 4 * lg;
    float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (bias) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (n + c < g.Nout) b[c] = T::lo(bias[n + c]);
    }
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
      const int m = wm * C::WTM + i * 16 + lr;
      if (m < mrows && n < g.Nout && (!SUMS || g.C)) {
        const v4f& x = acc[i][j];
        store4<T>(out + (uint64_t)(m0 + m) * g.Nout + n, n, g.Nout, x[0] + b[0], x[1] + b[1], x[2] + b[2], x[3] + b[3]);
      }
    }
  }
  if constexpr (SUMS)
    if (with_sums && lg == 0) {
#pragma unroll
      for (int i = 0; i < C::FM; ++i) {
        const int m = m0 + wm * C::WTM + i * 16 + lr;
        if (m < g.Mout) g.dbias[(uint64_t)e * g.Mout + m] = (uint16_t)T::pack(sums[i][0], 0.0f);
      }
    }
}

template <class C>
__global__ __launch_bounds__(C::NT, C::NW / 4 * (C::LDS > 80 * 1024 ? 1 : 2)) void sk_grouped(GroupedGemm g) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LDS];
  grouped_tile<C>(g, (lds_u8*)smem);
}

template <class C>
hipError_t launch_grouped_tiles(GroupedGemm g, hipStream_t s) {
  int64_t grid;
  if (C::KIND == kGradB) {
    g.tiles_m = cdiv(g.Mout, C::BM);
    g.tiles_n = g.C ? cdiv(g.Nout, C::BN) : 1;      // (dbias alone is made by the first column's tiles)
    grid = (int64_t)g.E * g.tiles_m * g.tiles_n;
  } else {
    // every group but one may end with a tile of one row
    const int groups = g.E + (g.tail ? 1 : 0);
    g.tiles_m = (int)(((int64_t)g.R + (int64_t)groups * (C::BM - 1)) / C::BM);
    g.tiles_n = cdiv(g.Nout, C::BN);
    grid = (int64_t)g.tiles_m * g.tiles_n;
  }
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  return launch(sk_grouped<C>, dim3((unsigned)grid), C::NT, s, g);
}

template <class T>
hipError_t launch_grouped_of(const GroupedGemm& g, int kind, int cus, hipStream_t s) {
  if (kind == kGradB) return launch_grouped_tiles<GroupedCfg<T, kGradB, 256, 256, 2, 2, 2>>(g, s);
  if (kind == kGradA) return launch_grouped_tiles<GroupedCfg<T, kGradA, 256, 256, 2, 2, 2>>(g, s);
  return launch_grouped_tiles<GroupedCfg<T, kForward, 256, 256, 2, 2, 2>>(g, s);
}

}  // namespace sk

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

// The two element types: the matrix instruction, and rounding.  (16 x 16 x 32 products, whose rate under the power limit is 10 %
// above that of 32 x 32 x 16 ones: 2094 against 1899 TFLOP/s on random operands.)
struct Bf16 {
  static __device__ __forceinline__ v4f mfma(v4u b, v4u a, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, b), __builtin_bit_cast(v8bf, a), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) { return pack_bf16(a, b); }
  static __device__ __forceinline__ float lo(uint32_t w) { return bf16_lo(w); }
  static __device__ __forceinline__ float hi(uint32_t w) { return bf16_hi(w); }
  static constexpr uint32_t kOnes = 0x3f803f80u, kMinus16 = 0xbb80bb80u, kMinus24 = 0xbbc0bbc0u;      // (by 2^-12: sk_rows.hip)
  // c plus both halves of w
  static __device__ __forceinline__ float add2(uint32_t w, float c) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2, w), __builtin_bit_cast(b2, kOnes), c, false);
  }
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
  static constexpr uint32_t kOnes = 0x3c003c00u, kMinus16 = 0xcc00cc00u, kMinus24 = 0xce00ce00u;
  static __device__ __forceinline__ float add2(uint32_t w, float c) {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(h2, w), __builtin_bit_cast(h2, kOnes), c, false);
  }
};

enum GroupedKind { kForward = 0, kGradA = 1, kGradB = 2 };

// Tile BM x BN of the output on WM x WN waves.  k-steps of 64 of the dimension summed over; LDS is a ring of SLOTS places, each for one
// operand's part of a k-step (P of step 0, Q of step 0, P of step 1, ...).
// GATHER: A's rows are chosen by `rows`.
template <class T_, int KIND_, bool GATHER_, int BM_, int BN_, int WM_, int WN_, int SLOTS_>
struct GroupedCfg {
  using T = T_;
  static constexpr bool GATHER = GATHER_;
  static constexpr int KIND = KIND_, BM = BM_, BN = BN_, WM = WM_, WN = WN_, SLOTS = SLOTS_;
  static constexpr int NW = WM * WN, NT = 64 * NW;
  static constexpr int WTM = BM / WM, WTN = BN / WN, FM = WTM / 16, FN = WTN / 16;
  static constexpr bool PT = KIND == kGradB, QT = KIND != kForward;   // operands to be turned
  static constexpr int P_PT = BM / 8 / NW, Q_PT = BN / 8 / NW, D = P_PT + Q_PT;   // direct loads of a wave and k-step
  static constexpr int SLOT = (BM > BN ? BM : BN) * 128, LDS = SLOTS * SLOT;
  // loads of the first n parts behind part `from`
  static constexpr int loads(int from, int n) { return n <= 0 ? 0 : (from % 2 ? Q_PT : P_PT) + loads(from + 1, n - 1); }
  static_assert(SLOTS >= 4, "a k-step that is read and the next one");
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "whole loads for each wave");
  static_assert(LDS <= 160 * 1024, "LDS");
};

// Direct-to-LDS loads of 16 bytes a lane to LDS address lds + IMM, of which the second kind first moves the scalar offset on: that addition
// is the wait state between the write of m0 and its use.  (Few instructions: a wave has to issue them in the 12 cycles that a
// 16 x 16 x 32 MFMA leaves it.)
template <uint32_t IMM>
__device__ __forceinline__ void dma16(const v4u& rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  dma_load16_at<IMM>(rsrc, voff, soff, lds);
}
template <uint32_t IMM>
__device__ __forceinline__ void dma16_next(const v4u& rsrc, uint32_t voff, uint32_t& soff, uint32_t step, uint32_t lds) {
  asm volatile("s_add_u32 m0, %2, %5\n\ts_add_u32 %0, %0, %4\n\tbuffer_load_dwordx4 %1, %3, %0 offen lds"
               : "+s"(soff)
               : "v"(voff), "s"(lds), "s"(rsrc), "s"(step), "n"(IMM)
               : "memory", "m0", "scc");
}

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
  // loads of a wave after which the permutation repeats: load i + ALIKE is NW ALIKE RPU rows on, the same otherwise
  static constexpr int PERIOD = 16;                                // rows
  static constexpr int ALIKE = NW * RPU % PERIOD == 0 ? 1 : PERIOD / (NW * RPU);
  static_assert(PERIOD % (NW * RPU) == 0 || NW * RPU % PERIOD == 0, "whole periods");
  static_assert(!TURN || BX == 128 || BX == 256, "the permutation below");

  // The permutation of a turned operand's row, in 16-byte chunks.
  static __device__ __forceinline__ int swizzle(int row) { return 2 * ((row & 3) | ((row >> 3) & 1) << 2); }
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

// A workgroup's tile, or one of the `pieces` (1, 2 or 4) that it is cut into.
struct GroupTile {
  int e;           // expert; E for the rows behind the last one's
  int row0, rows;  // the tile's rows
  int tn;          // its column of tiles
  int piece, pieces;
};

// The tile of workgroup t (false: none).  Groups in order, each in bands of BAND tile rows by all its columns, and the
// list of tiles cut into eight runs, one for each XCD (workgroups are dealt to them in turn), whose L2 then
// holds an expert's weights for several workgroups.  (8192^3, bands of 4: 803 us; of 2 806, of 8 823, all rows 1158.)
// The tiles that are left when every unit has had as many as all can have (rem of them) are cut into 2 (along the columns) or 4
// pieces if those still run at once.
template <int BM, int BAND>
__device__ __forceinline__ bool find_tile(const GroupedGemm& g, int t, GroupTile* out) {
  const int* const offsets = g.offsets;
  const int lane = threadIdx.x & 63, E = g.E, R = g.R, G = E + (g.tail ? 1 : 0), tiles_n = g.tiles_n;
  auto tiles_of = [&](int e) {
    int a = 0, b = 0;
    if (e < G) group_rows(offsets, e, E, R, &a, &b);
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
  for (int e = 64; e < G; e += 64) {
    int x = tiles_of(e + lane);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) x += __shfl_xor(x, d);
    total += __builtin_amdgcn_readfirstlane(x);
  }
  const int T = (int)min((int64_t)total * tiles_n, (int64_t)g.most);
  out->piece = 0;
  out->pieces = 1;
  if (g.cus) {
    const int full = T / g.cus * g.cus, rem = T - full;
    const int pieces = rem == 0 ? 1 : rem * 4 <= g.cus ? 4 : rem * 2 <= g.cus ? 2 : 1;
    if (t >= full && pieces > 1) {
      const int u = t - full;
      out->piece = u / rem;
      out->pieces = pieces;
      if (out->piece >= pieces) return false;
      t = full + u - out->piece * rem;
    }
  }
  if (t >= T) return false;
  const int x = t & 7, per = T >> 3, rest = T & 7;
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
  out->rows = __builtin_amdgcn_readfirstlane(min(BM, b - a - tm * BM));
  out->tn = __builtin_amdgcn_readfirstlane(tn);
  return in >= 0 && tm < tm_e && tn < tiles_n;      // (always, unless wrong offsets make the numbers of tiles pass 32 bits)
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

// What a workgroup computes: `rows` rows from row0 on of expert e, and the output's columns from n0 on; dB: its rows from m0
// on, summed over these rows.
struct GroupedPart {
  int e, row0, rows, m0, n0;
};

// P is the operand of the output's rows, Q that of its columns.
// SUMS: dB's tile also adds up its rows of dC.
template <class C, bool SUMS>
__device__ __forceinline__ void grouped_tile(const GroupedGemm& g, const GroupedPart& part, lds_u8* const smem) {
  using T = typename C::T;
  using OpP = Operand<C::BM, C::NW, C::PT>;
  using OpQ = Operand<C::BN, C::NW, C::QT>;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int wm = wave / C::WN, wn = wave % C::WN, lr = lane & 15, lg = lane >> 4;
  const uint32_t ring = (uint32_t)(uintptr_t)smem;
  const int e = part.e, row0 = part.row0, rows = part.rows, m0 = part.m0, n0 = part.n0;
  const bool zeros = C::KIND != kGradB && e >= g.E;
  const int steps = zeros ? 0 : ((C::KIND == kGradB ? rows : g.S) + 63) / 64;

  // ---- where the operands' loads come from: a lane's offsets (one where a wave's loads differ by whole rows of the same
  // permutation, which a scalar offset then carries; one each for gathered rows), and a resource
  constexpr int PV = C::KIND == kForward && C::GATHER ? C::P_PT : OpP::ALIKE, QV = OpQ::ALIKE;
  const uint32_t pp = (uint32_t)g.p_pitch, qp = (uint32_t)g.q_pitch;
  const uint64_t e_off = zeros ? 0 : (uint64_t)e;
  uint32_t pvoff[PV], qvoff[QV];
  v4u pr, qr;
#pragma unroll
  for (int i = 0; i < PV; ++i) pvoff[i] = (uint32_t)OpP::row_of(wave, i, lane) * pp + OpP::chunk_of(wave, i, lane) * 16;
#pragma unroll
  for (int i = 0; i < QV; ++i) qvoff[i] = (uint32_t)OpQ::row_of(wave, i, lane) * qp + OpQ::chunk_of(wave, i, lane) * 16;
  if constexpr (C::KIND == kForward) {
    if constexpr (C::GATHER) {
#pragma unroll
      for (int i = 0; i < PV; ++i) {
        const int r = min(OpP::row_of(wave, i, lane), rows - 1);
        const int t = zeros ? 0 : min(max(g.rows[row0 + r], 0), g.p_rows - 1);
        pvoff[i] = (uint32_t)t * pp + OpP::chunk_of(wave, i, lane) * 16;
      }
      pr = rsrc_words(g.P, (uint32_t)g.p_rows * pp);
    } else {
      pr = rsrc_words(g.P + (uint64_t)row0 * pp, (uint32_t)rows * pp);
    }
    qr = rsrc_words(g.Q + (e_off * g.Nout + n0) * qp, (uint32_t)min(C::BN, g.Nout - n0) * qp);
  } else if constexpr (C::KIND == kGradA) {
    pr = rsrc_words(g.P + (uint64_t)row0 * pp, (uint32_t)rows * pp);
  } else if constexpr (C::GATHER) {
    qr = rsrc_words(g.Q + n0 * 2, (uint32_t)g.q_rows * qp - (uint32_t)n0 * 2);
  }
  // (gather, dB) where the wave's TOK rows of each of AHEAD k-steps begin, one in each lane, out of range where there is no row.  The
  // rows' indexes are asked for AHEAD k-steps before, since the wait for them is also one for all direct loads before it.  (Asked for in
  // every k-step, as scalars, they made all waits for LDS reads wait for them: 8002 rows of 8 experts, 2048 x 4096, 17 % longer.)
  constexpr int TOK = C::KIND == kGradB && C::GATHER ? C::Q_PT * OpQ::RPU : 1, AHEAD = 64 / TOK;
  uint32_t held = 0;
  int asked = 0;
  auto row_at = [&](int s) { return (s + lane / TOK) * 64 + wave * TOK + lane % TOK; };
  auto ask = [&](int s) {
    const int b = row_at(s);
    if (b < rows) asked = g.rows[row0 + b];
  };
  auto take = [&](int s) { held = row_at(s) < rows ? (uint32_t)min(max(asked, 0), g.q_rows - 1) * qp : kOob; };
  // Rows of the k-step at s of a turned operand: `have` rows from `base` on.
  auto turned = [&](const uint8_t* base, uint32_t pitch, int col0, int have, int s) {
    // (said to be uniform: a value held to a range goes to vector registers otherwise)
    const int left = __builtin_amdgcn_readfirstlane(min(max(have - s * 64, 0), 64));
    const uint32_t bytes = left > 0 ? (uint32_t)left * pitch - (uint32_t)col0 * 2 : 0u;
    return rsrc_words(base + (uint64_t)(left > 0 ? s : 0) * 64 * pitch + (uint32_t)col0 * 2, bytes);
  };

  // The direct loads of an operand's part of k-step s, one at a time; past the last k-step every lane is out of range (zeros,
  // no traffic).  (The range check is on the lane's offset plus the scalar one.)
  uint32_t kp = 0, kq = 0;   // the scalar offsets: where the k-step starts in a row of an operand that is not turned, and the loads' rows
  auto aim_p = [&](int s) {
    if constexpr (C::PT) {
      pr = turned(g.P + (uint64_t)row0 * pp, pp, m0, rows, s);
      kp = 0;
    } else {
      kp = (uint32_t)s * 128u;
      if (s >= steps - 1) {   // the last k-step's part, or none
        const uint32_t have = s == steps - 1 ? (uint32_t)(g.S * 2) - kp : 0u;
#pragma unroll
        for (int i = 0; i < PV; ++i) pvoff[i] |= (uint32_t)OpP::chunk_of(wave, i, lane) * 16 < have ? 0u : kOob;
      }
    }
  };
  auto aim_q = [&](int s) {
    if constexpr (C::KIND == kGradA) {
      qr = turned(g.Q + e_off * g.S * qp, qp, n0, g.S, s);
      kq = 0;
    } else if constexpr (C::KIND == kGradB && C::GATHER) {
      if (s > 0 && s % AHEAD == 0) {
        take(s);
        ask(s + AHEAD);
      }
      kq = (uint32_t)(s % AHEAD) * TOK;     // (here: the lane that holds the k-step's first row)
    } else if constexpr (C::KIND == kGradB) {
      qr = turned(g.Q + (uint64_t)row0 * qp, qp, n0, rows, s);
      kq = 0;
    } else {
      kq = (uint32_t)s * 128u;
      if (s >= steps - 1) {
        const uint32_t have = s == steps - 1 ? (uint32_t)(g.S * 2) - kq : 0u;
#pragma unroll
        for (int i = 0; i < QV; ++i) qvoff[i] |= (uint32_t)OpQ::chunk_of(wave, i, lane) * 16 < have ? 0u : kOob;
      }
    }
  };
  const uint32_t pstep = (uint32_t)(OpP::ALIKE * C::NW * OpP::RPU) * pp, qstep = (uint32_t)(OpQ::ALIKE * C::NW * OpQ::RPU) * qp;
  // (place: with the wave's own kilobyte)
  auto load_p = [&](uint32_t place, auto lc) {
    constexpr int i = decltype(lc)::value, v = i % PV;
    constexpr uint32_t at = (uint32_t)i * C::NW * 1024u;
    if constexpr (i >= PV && v == 0) dma16_next<at>(pr, pvoff[v], kp, pstep, place);
    else dma16<at>(pr, pvoff[v], kp, place);
  };
  auto load_q = [&](uint32_t place, auto lc) {
    constexpr int i = decltype(lc)::value, v = i % QV;
    constexpr uint32_t at = (uint32_t)i * C::NW * 1024u;
    if constexpr (C::KIND == kGradB && C::GATHER) {
      // the wave's rows one behind the other: its load i has rows i RPU .. of them
      const int part = lane / (64 / OpQ::RPU), row = wave * TOK + i * OpQ::RPU + part;
      uint32_t from = (uint32_t)__builtin_amdgcn_readlane((int)held, (int)kq + i * OpQ::RPU);
#pragma unroll
      for (int j = 1; j < OpQ::RPU; ++j) from = part == j ? (uint32_t)__builtin_amdgcn_readlane((int)held, (int)kq + i * OpQ::RPU + j) : from;
      const int chunk = (lane % (OpQ::ROW / 16)) ^ OpQ::swizzle(row);
      dma16<(uint32_t)i * 1024u>(qr, from + (uint32_t)chunk * 16, 0u, place + (uint32_t)wave * (C::Q_PT - 1) * 1024u);
    } else if constexpr (i >= QV && v == 0) {
      dma16_next<at>(qr, qvoff[v], kq, qstep, place);
    } else {
      dma16<at>(qr, qvoff[v], kq, place);
    }
  };
  // Part n (P of step n / 2 or Q of it): aimed at once, loaded one load at a time.
  auto aim = [&](auto odd, int s) {
    if constexpr (decltype(odd)::value % 2) aim_q(s);
    else aim_p(s);
  };
  auto load = [&](auto odd, uint32_t place, auto lc) {
    if constexpr (decltype(odd)::value % 2) load_q(place, lc);
    else load_p(place, lc);
  };

  // ---- the k-steps
  v4f acc[C::FM][C::FN];
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) acc[i][j] = v4f{};
  // of row lr of every WN-th block (the waves of a row share them out), over the lane's part of the dimension summed over
  constexpr int NSUM = SUMS ? (C::FM + C::WN - 1) / C::WN : 1;
  float sums[NSUM];
#pragma unroll
  for (int i = 0; i < NSUM; ++i) sums[i] = 0.0f;

  v4u p[2][C::FM], q[2][C::FN];
  uint32_t lp, lq;
  auto aim_reads = [&](uint32_t at_p, uint32_t at_q) {
    lp = OpP::read_base(at_p, wm * C::WTM, lane);
    lq = OpQ::read_base(at_q, wn * C::WTN, lane);
  };
  // Read n of the FM + FN of a half, in the order in which the products need them.
  auto read = [&](auto hc, auto nc) {
    constexpr int h = decltype(hc)::value, n = decltype(nc)::value;
    if constexpr (n == 0) q[h][0] = OpQ::template read<h>(lq, 0);
    else if constexpr (n <= C::FM) p[h][n - 1] = OpP::template read<h>(lp, n - 1);
    else q[h][n - C::FM] = OpQ::template read<h>(lq, n - C::FM);
  };
  // The reads beside a half's products are begun in its first three quarters, so that they are there at its end.  The direct
  // loads go behind the products of its first half with 8 waves (spread over all of it, 4148 rows of 16 experts, 2051 x
  // 1288, took 5 % longer, in the second half 11 %), and are spread over all of it with 4.
  constexpr int NS = C::FM * C::FN, NR = C::FM + C::FN, NB = NS >= 8 ? NS * 3 / 4 : NS;
  constexpr auto place_of = [](int l, int n) { return C::NW == 8 ? 1 + l * NS / n / 2 : l * NS / n; };      // behind which product load l of n goes
  using std::integral_constant;

  if (steps > 0) {
    if constexpr (C::KIND == kGradB && C::GATHER) {
      ask(0);
      take(0);
      ask(AHEAD);
    }
    static_for<C::SLOTS - 1>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
      aim(ic, i / 2);
      static_for<(i % 2 ? C::Q_PT : C::P_PT)>([&](auto l) { load(ic, ring + i * C::SLOT + wave * 1024u, l); });
    });
    wait_vmcnt_n<C::loads(2, C::SLOTS - 3)>();
    lds_barrier();
    aim_reads(ring, ring + C::SLOT);
    static_for<NR>([&](auto n) { read(integral_constant<int, 0>{}, n); });
    // places of the k-step being multiplied
    uint32_t at_p = ring, at_q = ring + C::SLOT, late = ring + (C::SLOTS - 1) * C::SLOT + wave * 1024u;   // late: where the previous k-step's Q was
    constexpr integral_constant<int, C::SLOTS> part0;
    constexpr integral_constant<int, C::SLOTS + 1> part1;
    constexpr int L0N = C::SLOTS % 2 ? C::Q_PT : C::P_PT, L1N = C::D - L0N;      // loads of the two
    constexpr uint32_t over = C::SLOTS * C::SLOT;
    auto on = [&](uint32_t at) { return at + 2 * C::SLOT >= ring + over ? at + 2 * C::SLOT - over : at + 2 * C::SLOT; };
    for (int s = 0; s < steps; ++s) {
      // first half: its products, and the second half's reads beside them
      aim(part1, s + (C::SLOTS - 1) / 2);
      static_for<NS>([&](auto nc) {
        constexpr int n = decltype(nc)::value, i = n % C::FM, j = n / C::FM;
        acc[i][j] = T::mfma(q[0][j], p[0][i], acc[i][j]);
        constexpr int R0 = n < NB ? n * NR / NB : NR, R1 = n < NB ? (n + 1) * NR / NB : NR;
        static_for<R1 - R0>([&](auto k) { read(integral_constant<int, 1>{}, integral_constant<int, R0 + decltype(k)::value>{}); });
        static_for<L1N>([&](auto l) {
          if constexpr (place_of(decltype(l)::value, L1N) == n) load(part1, late, l);
        });
        __builtin_amdgcn_sched_barrier(0);
      });
      if constexpr (SUMS) {      // (on the ALU: MFMAs of ones would cost an eighth more of them)
        static_for<C::FM>([&](auto ic) {
          constexpr int i = decltype(ic)::value;
          if (wn == i % C::WN)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int c = 0; c < 4; ++c) sums[i / C::WN] = T::add2(p[h][i][c], sums[i / C::WN]);
        });
      }
      // the next k-step has arrived and this one has been read: its two places are free
      wait_vmcnt_n<C::loads(4, C::SLOTS - 4)>();
      lds_barrier();
      const uint32_t free0 = at_p + wave * 1024u;
      late = at_q + wave * 1024u;
      at_p = on(at_p);
      at_q = on(at_q);
      aim_reads(at_p, at_q);
      aim(part0, s + C::SLOTS / 2);
      static_for<NS>([&](auto nc) {
        constexpr int n = decltype(nc)::value, i = n % C::FM, j = n / C::FM;
        acc[i][j] = T::mfma(q[1][j], p[1][i], acc[i][j]);
        constexpr int R0 = n < NB ? n * NR / NB : NR, R1 = n < NB ? (n + 1) * NR / NB : NR;
        static_for<R1 - R0>([&](auto k) { read(integral_constant<int, 0>{}, integral_constant<int, R0 + decltype(k)::value>{}); });
        static_for<L0N>([&](auto l) {
          if constexpr (place_of(decltype(l)::value, L0N) == n) load(part0, free0, l);
        });
        __builtin_amdgcn_sched_barrier(0);
      });
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }

  // ---- outputs: the lane has row lr and columns 4 lg .. + 3 of each 16 x 16 block.  Each wave turns 16 rows at a time into whole
  // stretches of a row through LDS, 16 bytes to a lane (stored as they lie, 8 bytes to a lane in runs of 32, 4148 x 2048
  // outputs took 18 us and not 11, and dB of 8 x 2048 x 4096 70 us of 230).
  lds_barrier();      // every wave has read its last operands, and no direct load is under way
  const uint16_t* const bias = C::KIND == kForward && g.bias && !zeros ? g.bias + (uint64_t)e * g.Nout : nullptr;
  uint16_t* const out = C::KIND == kGradB ? g.C + (uint64_t)e * g.Mout * g.Nout : g.C + (uint64_t)row0 * g.Nout;
  const int mrows = C::KIND == kGradB ? min(C::BM, g.Mout - m0) : rows;
  if (!SUMS || g.C) {
    constexpr int CH = C::WTN / 8, RPL = 64 / CH;      // 16-byte chunks of a row; rows of a store
    int ln = lane;      // (a copy whose uses cannot move ahead of the k-steps, where there are no registers for them)
    asm volatile("" : "+v"(ln));
    const int lr = ln & 15, lg = ln >> 4;
    static_assert(CH == 8 || CH == 4, "the permutation below");
    auto turn = [](int row) { return CH == 8 ? (row >> 1) & 7 : (row >> 2) & 3; };   // of a row's chunks, for the banks
    const uint32_t area = ring + (uint32_t)wave * 16 * C::WTN * 2;
    const int nw = n0 + wn * C::WTN;
    float b[C::FN][4];
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int n = nw + j * 16 + 4 * lg + c;
        b[j][c] = C::KIND == kForward && bias && n < g.Nout ? T::lo(bias[n]) : 0.0f;
      }
    const int srow = ln / CH, schunk = ln % CH, sn = nw + schunk * 8;
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
#pragma unroll
      for (int j = 0; j < C::FN; ++j) {
        const v4f& x = acc[i][j];
        const uint32_t at = area + (uint32_t)(lr * C::WTN * 2 + (((2 * j + (lg >> 1)) ^ turn(lr)) * 16) + 8 * (lg & 1));
        *(__attribute__((address_space(3))) v2u*)(uintptr_t)at =
            v2u{T::pack(x[0] + b[j][0], x[1] + b[j][1]), T::pack(x[2] + b[j][2], x[3] + b[j][3])};
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
      for (int r = 0; r < 16; r += RPL) {
        const int row = r + srow, m = wm * C::WTM + i * 16 + row;
        const v4u v = *(const __attribute__((address_space(3))) v4u*)(uintptr_t)(area + (uint32_t)(row * C::WTN * 2 + ((schunk ^ turn(row)) * 16)));
        if (m < mrows && sn < g.Nout) {
          uint16_t* const to = out + (uint64_t)(m0 + m) * g.Nout + sn;
          if (sn + 8 <= g.Nout) {
            *(u32x4_any*)to = v;
          } else {
#pragma unroll
            for (int c = 0; c < 8; ++c)
              if (sn + c < g.Nout) to[c] = (uint16_t)(v[c / 2] >> (16 * (c & 1)));
          }
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
  }
  if constexpr (SUMS) {
#pragma unroll
    for (int n = 0; n < NSUM; ++n) {
      float x = sums[n];
      x += __shfl_xor(x, 16);
      x += __shfl_xor(x, 32);
      const int i = n * C::WN + wn, m = m0 + wm * C::WTM + i * 16 + lr;
      if (i < C::FM && lg == 0 && m < g.Mout) g.dbias[(uint64_t)e * g.Mout + m] = (uint16_t)T::pack(x, 0.0f);
    }
  }
}

// C: the tiles; H and Q: their halves and quarters.
template <class C, class H, class Q>
__global__ __launch_bounds__(C::NT, C::NW / 4 * (C::LDS > 80 * 1024 ? 1 : 2)) void sk_grouped(GroupedGemm g) {
  constexpr int LDS = C::LDS > Q::LDS ? C::LDS > H::LDS ? C::LDS : H::LDS : Q::LDS > H::LDS ? Q::LDS : H::LDS;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[LDS];
  GroupedPart p;
  if constexpr (C::KIND == kGradB) {
    // The experts in turn, and of each one's tiles (columns of them in turn) a run to each XCD.  (With a run of all experts' tiles
    // to each XCD, which leaves it with the experts that have the most rows, 8 experts of 500 to 1600 rows, 4096 x 2048, took
    // 28 % longer.  The experts with the most rows first: no change.)
    const int per_e = g.tiles_m * g.tiles_n, t = (int)blockIdx.x % per_e;
    p.e = (int)blockIdx.x / per_e;
    const int x = t & 7, i = x * (per_e >> 3) + min(x, per_e & 7) + (t >> 3), tn = i / g.tiles_m;
    p.m0 = (i - tn * g.tiles_m) * C::BM;
    p.n0 = tn * C::BN;
    int end;
    group_rows(g.offsets, p.e, g.E, g.R, &p.row0, &end);
    p.row0 = __builtin_amdgcn_readfirstlane(p.row0);
    p.rows = __builtin_amdgcn_readfirstlane(end) - p.row0;
    if (g.dbias && p.n0 == 0) grouped_tile<C, true>(g, p, (lds_u8*)smem);
    else grouped_tile<C, false>(g, p, (lds_u8*)smem);
  } else {
    GroupTile t;
    if (!find_tile<C::BM, C::BM >= 256 ? 4 : 8>(g, (int)blockIdx.x, &t)) return;
    p.e = t.e;
    p.row0 = t.row0;
    p.rows = t.rows;
    p.m0 = 0;
    p.n0 = t.tn * C::BN;
    if constexpr (!std::is_same_v<C, Q>) {
      if (t.pieces == 4) {
        p.row0 += t.piece / 2 * Q::BM;
        p.rows = min(Q::BM, p.rows - t.piece / 2 * Q::BM);
        p.n0 += t.piece % 2 * Q::BN;
        if (p.rows > 0 && p.n0 < g.Nout) grouped_tile<Q, false>(g, p, (lds_u8*)smem);
        return;
      }
      if (t.pieces == 2) {
        p.n0 += t.piece * H::BN;
        if (p.n0 < g.Nout) grouped_tile<H, false>(g, p, (lds_u8*)smem);
        return;
      }
    }
    grouped_tile<C, false>(g, p, (lds_u8*)smem);
  }
}

template <class C, class H, class Q>
hipError_t launch_grouped_tiles(GroupedGemm g, int cus, hipStream_t s) {
  int64_t grid;
  if (C::KIND == kGradB) {
    g.tiles_m = cdiv(g.Mout, C::BM);
    g.tiles_n = g.C ? cdiv(g.Nout, C::BN) : 1;      // (dbias alone is made by the first column's tiles)
    grid = (int64_t)g.E * g.tiles_m * g.tiles_n;
  } else {
    // every group but one may end with a tile of one row
    const int groups = g.E + (g.tail ? 1 : 0);
    g.tiles_n = cdiv(g.Nout, C::BN);
    grid = ((int64_t)g.R + (int64_t)groups * (C::BM - 1)) / C::BM * g.tiles_n;
    if (grid > 0x7fffffff) return hipErrorInvalidValue;
    g.most = (int)grid;
    g.cus = std::is_same_v<C, Q> ? 0 : cus;
    if (g.cus) grid += cus;         // at most so many more pieces than tiles
  }
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  return launch(sk_grouped<C, H, Q>, dim3((unsigned)grid), C::NT, s, g);
}

template <class T, int KIND, bool GATHER>
hipError_t launch_grouped_kind(const GroupedGemm& g, int cus, hipStream_t s) {
  // 8 waves, two to a SIMD, so that one's products hide the other's loads and reads: 4 waves of 128 x 128 each, which read a
  // third less from LDS, took 3 % longer for 4096 rows of 8 experts, 4096 x 4096, and 13 % for their dB with gathered rows.
  using Big = GroupedCfg<T, KIND, GATHER, 256, 256, 2, 4, 5>;
  using Half = GroupedCfg<T, KIND, GATHER, 256, 128, 2, 4, 5>;
  using Quarter = GroupedCfg<T, KIND, GATHER, 128, 128, 2, 4, 5>;
  using Small = GroupedCfg<T, KIND, GATHER, 128, 128, 2, 2, 5>;
  if constexpr (KIND == kGradB) {
    // (Here and below calls among others, with operands from memory.)  Smaller tiles read dC and A more often (8 experts of 2048 x 4096,
    // 8002 rows 128 us against 162 of 128 x 128), but are more where the large ones leave half of the units idle: 4 experts of
    // 1024 x 1024, 400 rows 8.7 / 6.3 and 1600 rows 14.8 / 10.2; of 2048 x 2048, 800 rows 15.7 / 17.4.
    if (g.E * (int64_t)cdiv(g.Mout, 256) * cdiv(g.Nout, 256) * 2 > cus) return launch_grouped_tiles<Big, Big, Big>(g, cus, s);
  } else {
    // about how many tiles there are with `rows` rows
    auto tiles = [&](int rows, int cols) { return ((int64_t)g.R / rows + g.E / 2) * cdiv(g.Nout, cols); };
    // Tiles of 256 x 256 where experts have 128 rows or more on the average and there are tiles for half of the units: 4096 x
    // 4096, 8 experts, 4096 rows 113 us against 157 of 128 x 128, 2048 rows 84 / 91, 1024 rows 72 / 68, 512 rows 67 / 65; dA of
    // 2048 rows 75 / 89, 1024 rows 65 / 58; 64 experts of 512 x 1024 with 125 rows each 23.4 / 21.2.
    if ((int64_t)g.R >= 128 * (int64_t)g.E && tiles(256, 256) * 2 >= cus) return launch_grouped_tiles<Big, Half, Quarter>(g, cus, s);
    // Tiles of 32 x 128, in which most rows are there, for up to 24 rows of an expert: 8 experts of 4096 x 4096, 8 rows 59.9 us
    // against 62.6 with 128 x 128 (the weights alone take 44 to 55), 512 rows 65.3 / 64.8, 1024 rows 115 / 68; 64 experts of 2048 x 1024 with
    // 28 rows each 61.9 / 56.0.  And where all of them run at once, since a k-step of one takes half the time: 4 experts of 1024 x
    // 1024, 800 rows 9.3 us against 16.1, 1600 rows 17.1 / 16.2.
    using Few = GroupedCfg<T, KIND, GATHER, 32, 128, 1, 4, 8>;
    if ((int64_t)g.R <= 24 * (int64_t)g.E || tiles(32, 128) <= cus) return launch_grouped_tiles<Few, Few, Few>(g, cus, s);
    // Of 64 x 128 by the same rule: 4 experts of 1024 x 1024, 1600 rows 10.7 us against 16.2 with 128 x 128, of 2048 x 2048, 800 rows
    // 18.0 / 28.5 and 1200 rows 33.4 / 28.6.
    using Mid = GroupedCfg<T, KIND, GATHER, 64, 128, 2, 2, 8>;
    if (tiles(64, 128) <= cus) return launch_grouped_tiles<Mid, Mid, Mid>(g, cus, s);
  }
  return launch_grouped_tiles<Small, Small, Small>(g, cus, s);
}

template <class T>
hipError_t launch_grouped_of(const GroupedGemm& g, int kind, int cus, hipStream_t s) {
  if (kind == kGradA) return launch_grouped_kind<T, kGradA, false>(g, cus, s);
  if (kind == kGradB) return g.rows ? launch_grouped_kind<T, kGradB, true>(g, cus, s) : launch_grouped_kind<T, kGradB, false>(g, cus, s);
  return g.rows ? launch_grouped_kind<T, kForward, true>(g, cus, s) : launch_grouped_kind<T, kForward, false>(g, cus, s);
}

}  // namespace sk

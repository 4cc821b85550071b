// The product of E4M3 operands with an fp32 scale for each block of 128 along K:
//
//   C[m][n] = bf16( sum_b SA[b][m] SB(b, n) sum_{k in b} A[m][k] B[n][k] + bias[n] )
//
// SB(b, n) is a scale of its own for each row of B, [b][n], or one for 128 rows, [n / 128][b].  A block's
// inner sum is one v_mfma_f32_16x16x128_f8f6f4 from a zero accumulator; its 16 x 16 result is multiplied by
// the scales and added to the fp32 accumulators on the vector ALU (they change from block to block, so the
// MFMA cannot carry them, and its own scale operands are powers of two).  That is one fma per output and
// block (and one product of the two scales more where B has a scale per row): 4 x 4 cycles beside an MFMA of
// 32, issued by the same SIMD while the matrix core runs.
//
// Tiled kernels: k-steps of one block.  A's and B's 128 bytes per row and the step's scales go straight from
// memory into LDS (16-byte and 4-byte direct loads), in a ring of STAGES; the 16-byte chunks of row r are
// permuted by (r >> 1) & 7 so that 16 lanes reading a chunk of 16 rows meet all banks.  The accumulators are
// ordinary registers (the ALU cannot reach AGPRs), which bounds a wave's tile to 64 x 128.
// 8192^3: 422-460 us on different devices (2.4-2.6 PFLOP/s), 340 us on operands of zeros: held by power.  4096^3 60 us,
// 70 us with a scale per row of B: the second product per output and block fills the ALU.
// Few outputs: see sk_gemm_block_rows.

#include "sk_fp8.h"
#include "sk_kernel.h"

namespace sk {

namespace {

// A tile's 128-byte k-step of BM rows of A and BN of B over WM x WN waves; WK such groups of waves take every WK-th
// block of K, each with a ring of its own, and their sums are added in group order at the end.
template <int BM_, int BN_, int WM_, int WN_, int STAGES_, int WK_ = 1, bool STREAM_ = false>
struct BlockCfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, STAGES = STAGES_, WK = WK_;
  static constexpr int NW = WM * WN, NT = 64 * NW * WK;             // waves of a group, threads of a workgroup
  static constexpr int WTM = BM / WM, WTN = BN / WN;
  static constexpr int FM = WTM / 16, FN = WTN / 16;
  static constexpr int A_PT = BM / 8 / NW, B_PT = BN / 8 / NW;      // 1 KiB loads (8 rows) per wave
  static constexpr int S_A = (BM + 63) / 64, S_B = (BN + 63) / 64;  // 256-byte scale loads of a stage
  static constexpr int S_PT = (S_A + S_B + NW - 1) / NW;            // ... per wave (past the last, one again)
  static constexpr int PER_STAGE = A_PT + B_PT + S_PT;
  // Two stages: A's part of one, which is in registers by then, is refilled during the k-step that uses it, behind a
  // barrier of its own (see the k-steps).  Needs three pairs of columns.
  static constexpr bool EARLY_A = STAGES == 2 && FN > 4;
  static constexpr int B_OFF = BM * kBlock, S_OFF = (BM + BN) * kBlock, SB_OFF = S_OFF + S_A * 256;
  static constexpr int STAGE = SB_OFF + S_B * 256;
  // Outputs leave through LDS, a wave's OR rows at a time: all of them where the ring is done with.  Where a
  // workgroup takes several tiles (STREAM) the next tile's first stages are on their way into the ring by then,
  // and the outputs have a small area of their own.  (Whole rows of a wave all the same: half of them, 128 bytes that
  // start anywhere, are mostly lines written in part, 5000x6001x700 40.6 -> 48.5 us.)
  static constexpr bool STREAM = STREAM_;
  static constexpr int OR = STREAM ? 8 : WTM, OUT_WAVE = OR * WTN * 2;
  static constexpr int CH = WTN / 8;                                // 16-byte chunks of an output row
  static constexpr int RING = STAGES * STAGE, BIAS = BN < 128 ? 256 : 2 * BN, BIAS_OFF = WK * RING;
  static constexpr int OUT_OFF = STREAM ? BIAS_OFF + 2 * BIAS : 0;
  static constexpr int LDS = STREAM ? OUT_OFF + NW * OUT_WAVE : BIAS_OFF + BIAS;
  static_assert(A_PT * NW * 8 == BM && B_PT * NW * 8 == BN, "whole loads");
  static_assert(WTM % 16 == 0 && WTN % 16 == 0 && WTN <= 128 && 128 % WTN == 0, "a wave's columns share a tile scale");
  static_assert(NW * OUT_WAVE <= BIAS_OFF && LDS <= 160 * 1024, "LDS");
  static_assert(!STREAM || (WK == 1 && BN <= 256 && BN / 128 <= NW), "a streamed tile");
  static_assert((STAGES - 1) * PER_STAGE + A_PT <= 63, "vmcnt range");
  static_assert(WK == 1 || NW * OUT_WAVE + (WK - 1) * BM * BN * 4 <= BIAS_OFF, "sums passed between the groups");
};

// Tile t of the launch as (tile row, tile column): workgroups are dealt to the eight XCDs in turn, so each
// XCD gets a contiguous range of tiles, and within it patches of GROUP tile rows by whole columns,
// whose operands its L2 then holds for several workgroups.
template <int GROUP>
__device__ __forceinline__ void tile_of(int t, int tiles_m, int tiles_n, int* tm, int* tn) {
  const int T = tiles_m * tiles_n, x = t & 7, per = T >> 3, rest = T & 7;
  const int i = x * per + min(x, rest) + (t >> 3);
  const int band = i / (GROUP * tiles_n), in = i - band * GROUP * tiles_n;
  const int rows = min(GROUP, tiles_m - band * GROUP);
  *tn = in / rows;
  *tm = band * GROUP + (in - *tn * rows);
}

// A value that is the same in every lane, said so (a choice between 64-bit values goes to vector registers otherwise).
__device__ __forceinline__ int64_t uniform(int64_t x) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)x);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(x >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// One block's inner products, transposed as elsewhere here (B first): lane l gets A row l % 16 and the four
// B rows 4 (l / 16) .. +3.  The operand order within the 128 elements is the same for both, so any will do.
__device__ __forceinline__ v4f block_mfma(const v4u (&b)[2], const v4u (&a)[2]) {
  auto v = [](const v4u(&x)[2]) {
    return v8i{(int)x[0][0], (int)x[0][1], (int)x[0][2], (int)x[0][3],
               (int)x[1][0], (int)x[1][1], (int)x[1][2], (int)x[1][3]};
  };
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v(b), v(a), v4f{}, FMT_E4M3, FMT_E4M3, 0, 0, 0, 0);
}

__device__ __forceinline__ v4f ld_v4f(const lds_u8* p) { return *(const __attribute__((address_space(3))) v4f*)p; }
__device__ __forceinline__ v4u ld_v4u(const lds_u8* p) { return *(const __attribute__((address_space(3))) v4u*)p; }

// out[n] = bf16 of the sum of part's rows at column n, in an order that does not depend on NT: slice k of kSumSlices
// adds its run of rows in turn, then the runs are added in turn.  A workgroup takes NT / kSumSlices columns.
constexpr int kSumSlices = 16;
template <int NT>
__device__ __forceinline__ void column_sums_bf16(const ColumnSums& c, int block, float* run) {
  constexpr int COLS = NT / kSumSlices;
  const int col = threadIdx.x % COLS, slice = threadIdx.x / COLS, n = block * COLS + col;
  const int per = (c.count + kSumSlices - 1) / kSumSlices, c0 = slice * per, c1 = min(c.count, c0 + per);
  float s = 0.0f;
  if (n < c.N) {
#pragma unroll 4
    for (int r = c0; r < c1; ++r) s += c.part[(int64_t)r * c.N + n];
  }
  run[threadIdx.x] = s;
  __syncthreads();
  if (slice || n >= c.N) return;
  float x = run[col];
#pragma unroll
  for (int k = 1; k < kSumSlices; ++k) x += run[k * COLS + col];
  c.out[n] = (uint16_t)pack_bf16(x, x);
}

// Four outputs of a row: sums plus bias, rounded once to bf16 (the sum with the bias is one more fp32 addition).
__device__ __forceinline__ v2u out4(const v4f& x, const float (&b)[4]) {
  return v2u{pack_bf16(x[0] + b[0], x[1] + b[1]), pack_bf16(x[2] + b[2], x[3] + b[3])};
}

// Tiles first, first + stride, ... of one product.
template <class C, bool BROW>
__device__ __forceinline__ void block_tiles(const BlockGemm& g, lds_u8* const smem, int first, int stride) {
  const int lane = threadIdx.x & 63, wave = wave_id() % C::NW, group = wave_id() / C::NW;
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int lr = lane & 15, lg = lane >> 4;
  const uint32_t rb = (uint32_t)g.row_bytes;
  const uint32_t ring = (uint32_t)(uintptr_t)smem + (uint32_t)group * C::RING;
  const int steps = (g.kb + C::WK - 1) / C::WK;          // k-steps; step d of a group is block d WK + group

  // The lane's part of a direct load: slot lane % 8 of row lane / 8 of an 8-row group.  A wave's next group is NW
  // of them on: whole 16-row periods, the same chunk again, or with one wave half a period, the chunk 64 bytes away.
  const int grow = wave * 8 + (lane >> 3);
  const uint32_t chunk = (uint32_t)(((lane & 7) ^ ((grow >> 1) & 7)) * 16);
  const uint32_t row_off = (uint32_t)grow * rb;
  const uint32_t gstep = (uint32_t)(C::NW * 8) * rb;     // to the wave's next group, in the scalar offset

  // The lane's operand chunks lg and 4 + lg of row lr of each 16-row block.  (Any four a half will do that are the
  // same for A and B; a 16-byte read serves lanes 0-3, 12-15, 20-23 and 24-27 together, then the four other
  // quads, so lane groups 0 and 1 have to differ in the chunk's lowest bit: chunks 2 lg, 2 lg + 1 met
  // every bank twice.)
  const int sw = (lr >> 1) & 7;
  const int c0 = (lg ^ sw) * 16;

  const int T = g.tiles_m * g.tiles_n;
  // The tile that loads are issued for.  This wave's scale loads of a stage are 64 floats each: rows of A, or columns of B,
  // whose scale is their own or that of their 128 columns.  The k-steps are issued in order: sat is where the next
  // one's are, sstep bytes on from the last block's.
  int m0, n0, rows, cols;
  v4u ra, rbw;
  int64_t sat[C::S_PT], sstep[C::S_PT];
  uint32_t sbytes[C::S_PT], svoff[C::S_PT], slds[C::S_PT];
  // the tile's bias goes to LDS too, two columns a lane (a lone last column, or a bias not on four bytes, would
  // not: it is read when the outputs are made)
  const bool bias_staged = (((uintptr_t)g.bias | (uintptr_t)(2 * g.N)) & 3) == 0;
  constexpr int BI = (C::BN + 127) / 128;
  auto aim = [&](int t, int turn) {
    int tm, tn;
    tile_of<C::BM >= 256 ? 4 : 8>(t, g.tiles_m, g.tiles_n, &tm, &tn);
    tm = __builtin_amdgcn_readfirstlane(tm);
    tn = __builtin_amdgcn_readfirstlane(tn);
    m0 = tm * C::BM;
    n0 = tn * C::BN;
    rows = min(C::BM, g.M - m0);
    cols = min(C::BN, g.N - n0);
    ra = rsrc_words(g.A + (int64_t)m0 * rb, (uint32_t)rows * rb);
    rbw = rsrc_words(g.B + (int64_t)n0 * rb, (uint32_t)cols * rb);
#pragma unroll
    for (int i = 0; i < C::S_PT; ++i) {
      const int idx = (wave + i * C::NW) % (C::S_A + C::S_B);
      const bool is_a = idx < C::S_A;
      const int e = (is_a ? idx : idx - C::S_A) * 64 + lane, nb = n0 % kBlock;
      const float* const from = is_a ? g.SA + m0 : BROW ? g.SB + n0 : g.SB + (int64_t)(n0 / kBlock) * g.kb;
      sstep[i] = 4 * uniform(is_a ? g.M : BROW ? g.N : 1);
      sat[i] = uniform((int64_t)(uintptr_t)from) + group * sstep[i];
      sbytes[i] = (uint32_t)uniform(is_a ? rows : BROW ? cols : g.kb * ((nb + cols - 1) / kBlock + 1)) * 4u;
      svoff[i] = e >= (is_a ? rows : cols) ? kOob : (uint32_t)(is_a || BROW ? e : (nb + e) / kBlock * g.kb) * 4u;
      slds[i] = C::S_OFF + (uint32_t)idx * 256u;
    }
    if (bias_staged)
      dma_load4(rsrc_words(g.bias + n0, g.bias ? (uint32_t)cols * 2u : 0u), (uint32_t)((wave % BI) * 64 + lane) * 4u, 0u,
                (uint32_t)(uintptr_t)smem + C::BIAS_OFF + (uint32_t)turn * C::BIAS + (uint32_t)(wave % BI) * 256u);
  };
  // Load l of block k of that tile into a stage; where there is none every lane is out of range (zeros, no traffic).
  // (The range check is on the lane's offset plus the scalar one, measured also where the scalar one alone is past the end: row
  // groups beyond a ragged tile's rows read zeros.)
  auto issue_one = [&](int k, int slot, bool live, auto lc) {
    constexpr int l = decltype(lc)::value;
    const uint32_t stage = ring + (uint32_t)slot * C::STAGE;
    const uint32_t kbyte = live ? (uint32_t)k * kBlock : 0u;
    if constexpr (l < C::A_PT + C::B_PT) {
      constexpr bool is_a = l < C::A_PT;
      constexpr int i = is_a ? l : l - C::A_PT;
      const uint32_t c = chunk ^ (C::NW % 2 && i % 2 ? 64u : 0u);
      const uint32_t voff = live && kbyte + c < rb ? row_off + c : kOob;
      dma_load16(is_a ? ra : rbw, voff, kbyte + i * gstep,
                 stage + (is_a ? 0u : C::B_OFF) + (uint32_t)(wave + i * C::NW) * 1024u);
    } else {
      constexpr int i = l - C::A_PT - C::B_PT;
      dma_load4(rsrc_words((const void*)(uintptr_t)sat[i], sbytes[i]), live ? svoff[i] : kOob, 0u, stage + slds[i]);
      sat[i] += live ? C::WK * sstep[i] : 0;
    }
  };
  // Waves of a group meet (one alone only waits for its own LDS reads)
  auto meet = [&]() {
    if constexpr (C::NW > 1) lds_barrier();
    else asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  };

  // The k-steps as one stream of FM x FN slots, each starting a block's MFMA and adding the result of LAG slots
  // before, so that the ALU does not wait for the MFMA just started.  Columns of blocks go in pairs,
  // (i, j), (i, j + 1), (i + 1, j), ...: A's fragment i is used twice in a row, which spreads its refill for
  // the next stage (in place, after its last use) over the whole last pair of a k-step, and its first
  // use there over the whole first pair.  B's fragments go round a ring of two pairs, each read
  // during the pair before.  At the last pair every read of the stage has been issued: there the
  // waves wait for the next stage's loads (a whole k-step old) and meet, the loads of the stage after
  // go out into the one just read, and the reads run on into the next stage.  (EARLY_A: A's go out during the second
  // pair already, when every wave has its fragments, so that they have nearly two k-steps to arrive: with
  // two stages of 64 KiB the loads alone took as long as the k-step, 1.39 us, and 4096^3 65 us; now 61.)
  // sched_barrier(0) keeps the slots, and each MFMA before its slot's fmas, in this order.
  constexpr int NP = C::FN / 2, PS = 2 * C::FM, NS = C::FM * C::FN, LAG = 2;   // pairs; slots of a pair, of a k-step
  constexpr int RING = NP == 1 ? 2 : 4;
  static_assert(C::FN % 2 == 0 && (NP == 1 || NP % 2 == 0) && C::FM >= 2, "pairs of columns");
  v4u a[C::FM][2], b[RING][2];   // column j in b[j % RING]
  v4f sbv[RING];                 // (BROW) the four columns' scales
  float sa[C::FM], sbt = 0.0f;
  // LDS addresses in the stage being read, moved on behind each barrier.  (Chunk 4 + lg is 64 bytes from chunk lg,
  // with the sign of one of the permutation's bits: an exclusive or, since rows are 128 bytes.)
  uint32_t la, lb, lsa, lsb;
  auto aim_reads = [&]() {
    la = ring + (wm * C::WTM + lr) * kBlock + c0;
    lb = ring + C::B_OFF + (wn * C::WTN + lr) * kBlock + c0;
    lsa = ring + C::S_OFF + (wm * C::WTM + lr) * 4;
    lsb = ring + C::SB_OFF + (wn * C::WTN + (BROW ? 4 * lg : 0)) * 4;
  };
  auto at = [](uint32_t x) { return (const lds_u8*)(uintptr_t)x; };
  auto read_a = [&](auto ic) {
    constexpr int i = decltype(ic)::value;
    a[i][0] = ld_v4u(at(la) + i * 16 * kBlock);
    a[i][1] = ld_v4u(at(la ^ 64u) + i * 16 * kBlock);
  };
  auto read_b = [&](auto jc) {
    constexpr int j = decltype(jc)::value;
    b[j % RING][0] = ld_v4u(at(lb) + j * 16 * kBlock);
    b[j % RING][1] = ld_v4u(at(lb ^ 64u) + j * 16 * kBlock);
  };
  auto read_sb = [&](auto jc) {
    constexpr int j = decltype(jc)::value;
    if constexpr (BROW) sbv[j % RING] = ld_v4f(at(lsb) + j * 64);
  };
  auto read_scales = [&]() {
#pragma unroll
    for (int i = 0; i < C::FM; ++i) sa[i] = *(const __attribute__((address_space(3))) float*)(at(lsa) + i * 64);
    if constexpr (!BROW) sbt = *(const __attribute__((address_space(3))) float*)at(lsb);
  };

  // STREAM: one tile's loads follow the other's without a gap, so that no tile waits for its first stages or for the
  // stores of the last.  Takes more than STAGES k-steps a tile: the bias of tile t + 1 goes to the place of
  // tile t - 1's, which every wave has read once it has met the others in tile t's first k-step.
  int turn = 0;      // of the bias: tiles alternate
  int g0 = 0;        // k-steps before the tile's
  for (int t = first; t < T; t += stride) {
    const bool more = C::STREAM && t + stride < T;
    if (!C::STREAM || t == first) aim(t, turn);
    const int tm0 = m0, tn0 = n0, trows = rows, tcols = cols;     // the tile that is computed

    v4f acc[C::FM][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j) acc[i][j] = v4f{};

    if (!C::STREAM || t == first) {
#pragma unroll
      for (int d = 0; d < C::STAGES; ++d)
        static_for<C::PER_STAGE>([&](auto lc) { issue_one(d * C::WK + group, d, d * C::WK + group < g.kb, lc); });
      wait_vmcnt_n<(C::STAGES - 1) * C::PER_STAGE>();
      meet();
      aim_reads();
      read_scales();
      static_for<C::FM>(read_a);
      static_for<2>(read_b);
      static_for<2>(read_sb);
    }
    for (int d = 0; d < steps; ++d) {
      const int slot = (C::STREAM ? g0 + d : d) % C::STAGES;
      const int ahead = d + C::STAGES, ik = C::STREAM && ahead >= steps ? ahead - steps : ahead * C::WK + group;
      const bool live = C::STREAM ? ahead < steps || more : ik < g.kb;
      if constexpr (C::STREAM) {
        if (ahead == steps && more) aim(t + stride, turn ^ 1);     // from here on the loads are the next tile's
      }
      float s[C::FM];
#pragma unroll
      for (int i = 0; i < C::FM; ++i) s[i] = BROW ? sa[i] : sa[i] * sbt;
      v4f p[LAG + 1];
      auto add = [&](auto nc) {
        constexpr int n = decltype(nc)::value, i = n % PS / 2, j = n / PS * 2 + n % 2;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          acc[i][j][k] = __builtin_fmaf(BROW ? s[i] * sbv[j % RING][k] : s[i], p[n % (LAG + 1)][k], acc[i][j][k]);
      };
      static_for<NS>([&](auto nc) {
        constexpr int n = decltype(nc)::value, r = n % PS, i = r / 2, pair = n / PS, j = pair * 2 + n % 2;
        if constexpr (r == 0 && pair == NP - 1) {
          wait_vmcnt_n<(C::STAGES - 2) * C::PER_STAGE + (C::EARLY_A ? C::A_PT : 0)>();
          meet();
          const uint32_t move = (uint32_t)(slot + 1 < C::STAGES ? C::STAGE : -(C::STAGES - 1) * C::STAGE);
          la += move;
          lb += move;
          lsa += move;
          lsb += move;
          read_scales();   // (first: everything read later may still be on its way when the next k-step starts)
        }
        if constexpr (C::EARLY_A && r == 0 && pair == 1) meet();
        p[n % (LAG + 1)] = block_mfma(b[j % RING], a[i]);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (n >= LAG) add(std::integral_constant<int, n - LAG>{});
        // the next pair's columns, once the last pair's are done with (a stage of one pair: in place)
        if constexpr (NP > 1 && (r == 2 || r == 3)) {
          read_b(std::integral_constant<int, (j + 2) % C::FN>{});
          read_sb(std::integral_constant<int, (j + 2) % C::FN>{});
        }
        if constexpr (NP == 1 && i == C::FM - 1) read_b(std::integral_constant<int, j>{});
        if constexpr (pair == NP - 1) {
          if constexpr (n % 2 == 1) read_a(std::integral_constant<int, i>{});
          constexpr int early = C::EARLY_A ? C::A_PT : 0, count = C::PER_STAGE - early;
          static_for<count>([&](auto lc) {
            constexpr int l = decltype(lc)::value;
            if constexpr (l * PS / count == r) issue_one(ik, slot, live, std::integral_constant<int, early + l>{});
          });
        }
        if constexpr (C::EARLY_A && pair == 1) {
          static_for<C::A_PT>([&](auto lc) {
            constexpr int l = decltype(lc)::value;
            if constexpr (l * PS / C::A_PT == r) issue_one(ik, slot, live, lc);
          });
        }
        __builtin_amdgcn_sched_barrier(0);
      });
      static_for<LAG>([&](auto lc) { add(std::integral_constant<int, NS - LAG + decltype(lc)::value>{}); });
      if constexpr (NP == 1) static_for<2>(read_sb);
    }

    // outputs: each wave's through its own part of LDS, so that a store fills whole lines.  (The lane is read
    // afresh: offsets worked out from it would otherwise be kept, in spilled registers, through every k-step.)
    if constexpr (!C::STREAM) {
      wait_vmcnt_n<0>();
      lds_barrier();
    }
    int ol = lane;
    asm volatile("" : "+v"(ol));
    const int olr = ol & 15, olg = ol >> 4;
    if constexpr (C::WK > 1) {
      // the other groups' sums through LDS (behind the output staging), added in group order by the first, which stores
      lds_u8* const red = smem + C::NW * C::OUT_WAVE + (wave * C::FM * C::FN * 64 + lane) * 16;
      if (group > 0) {
        static_for<C::FM * C::FN>([&](auto nc) {
          constexpr int n = decltype(nc)::value;
          *(__attribute__((address_space(3))) v4f*)(red + (group - 1) * (C::BM * C::BN * 4) + n * 1024) =
              acc[n / C::FN][n % C::FN];
        });
      }
      lds_barrier();
      if (group == 0) {
        static_for<C::FM * C::FN>([&](auto nc) {
          constexpr int n = decltype(nc)::value;
#pragma unroll
          for (int k = 1; k < C::WK; ++k)
            acc[n / C::FN][n % C::FN] += ld_v4f(red + (k - 1) * (C::BM * C::BN * 4) + n * 1024);
        });
      }
    }
    const uint32_t so = (uint32_t)(uintptr_t)smem + C::OUT_OFF + wave * C::OUT_WAVE;
    auto finish = [&]() {
      v2u bias[C::FN];
      if (bias_staged) {
        const lds_u8* const at_bias = smem + C::BIAS_OFF + turn * C::BIAS + (wn * C::WTN + 4 * olg) * 2;
#pragma unroll
        for (int j = 0; j < C::FN; ++j) bias[j] = *(const __attribute__((address_space(3))) v2u*)(at_bias + j * 32);
      } else {
        const __amdgpu_buffer_rsrc_t rbias = make_rsrc(g.bias + tn0, g.bias ? (uint32_t)tcols * 2u : 0u);
#pragma unroll
        for (int j = 0; j < C::FN; ++j) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = __builtin_amdgcn_raw_buffer_load_b16(rbias, (uint32_t)(wn * C::WTN + j * 16 + 4 * olg + k) * 2u, 0, 0);
          bias[j] = v2u{w[0] | (w[1] << 16), w[2] | (w[3] << 16)};
        }
      }
      constexpr int RPI = 64 / C::CH;  // rows per store
      const int c = ol % C::CH, col = tn0 + wn * C::WTN + c * 8, orow = wm * C::WTM + ol / C::CH;
      const __amdgpu_buffer_rsrc_t rc = make_rsrc(g.C + (int64_t)tm0 * g.N, (uint32_t)trows * (uint32_t)g.N * 2u);
      // chunk q of row r is at (q ^ r) % CH.  Block j's chunks are 2 j and 2 j + 1: an exclusive or of 32 j bytes away
      // from block 0's (a row is a power of two, and starts at a multiple of itself).
      constexpr uint32_t PITCH = C::WTN * 2;
      static_assert((PITCH & (PITCH - 1)) == 0 && C::OUT_OFF % PITCH == 0 && C::OUT_WAVE % PITCH == 0 && PITCH <= 256, "rows");
      const int wrow = olr & (C::OR - 1);
      const uint32_t put = so + wrow * PITCH + ((((olg >> 1) ^ wrow) & (C::CH - 1)) * 16) + (olg & 1) * 8;
#pragma unroll
      for (int part = 0; part < C::WTM; part += C::OR) {
#pragma unroll
        for (int j = 0; j < C::FN; ++j) {
          const float b4[4] = {bf16_lo(bias[j][0]), bf16_hi(bias[j][0]), bf16_lo(bias[j][1]), bf16_hi(bias[j][1])};
#pragma unroll
          for (int i = part / 16; i < (part + C::OR + 15) / 16; ++i) {
            const v2u x = out4(acc[i][j], b4);
            if (C::OR >= 16 || olr / C::OR == part % 16 / C::OR)
              *(__attribute__((address_space(3))) v2u*)(uintptr_t)((put ^ (32u * j)) + (C::OR >= 16 ? (i * 16 - part) * PITCH : 0)) = x;
          }
        }
        asm volatile("" ::: "memory");   // (one wave's LDS operations execute in order)
        auto take = [&](int r0) {
          const int row = r0 + ol / C::CH;
          return ld_v4u(at(so + row * PITCH + ((c ^ (row & (C::CH - 1))) * 16)));
        };
        if ((g.N & 7) == 0) {
          const uint32_t to = ((uint32_t)(orow + part) * (uint32_t)g.N + (uint32_t)col) * 2u;
#pragma unroll
          for (int r0 = 0; r0 < C::OR; r0 += RPI)
            __builtin_amdgcn_raw_buffer_store_b128(take(r0), rc, col < g.N ? to + (uint32_t)r0 * (uint32_t)g.N * 2u : kOob, 0, 0);
        } else {
          // rows that start anywhere: the same sixteen bytes to any element's address, the row's last piece by elements
          uint16_t* const to = g.C + (int64_t)(tm0 + orow + part) * g.N + col;
#pragma unroll
          for (int r0 = 0; r0 < C::OR; r0 += RPI) {
            const v4u v = take(r0);
            if (orow + part + r0 >= trows) continue;
            uint16_t* const p = to + (int64_t)r0 * g.N;
            if (col + 8 <= g.N) {
              *(u32x4_any*)p = v;
            } else {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                if (col + k < g.N) p[k] = (uint16_t)(v[k / 2] >> (16 * (k & 1)));
            }
          }
        }
        asm volatile("" ::: "memory");
      }
    };
    if (group == 0) finish();
    if constexpr (C::STREAM) {
      g0 = (g0 + steps) % C::STAGES;
      turn ^= 1;
    } else if (t + stride < T) {
      lds_barrier();   // the next tile's loads go where the outputs were read from
    }
  }
  if constexpr (C::STREAM) wait_vmcnt_n<0>();     // nothing may still be on its way into LDS when the workgroup's is given up
}

template <class C, bool BROW>
__global__ __launch_bounds__(C::NT) void sk_gemm_block(BlockGemm g) {
  __shared__ __attribute__((aligned(256))) uint8_t smem[C::LDS];
  block_tiles<C, BROW>(g, (lds_u8*)smem, blockIdx.x, gridDim.x);
}

// The two products of a backward and the last pass of its column sums as one launch: the second product's tiles start
// as the first's end, and a small problem's three parts run side by side.
template <class C>
__global__ __launch_bounds__(C::NT) void sk_gemm_block_pair(BlockGemm a, BlockGemm b, ColumnSums c) {
  __shared__ __attribute__((aligned(256))) uint8_t smem[C::LDS];
  const int ta = a.tiles_m * a.tiles_n, tb = b.tiles_m * b.tiles_n, wg = blockIdx.x;
  if (wg < ta) block_tiles<C, false>(a, (lds_u8*)smem, wg, ta);
  else if (wg < ta + tb) block_tiles<C, true>(b, (lds_u8*)smem, wg - ta, tb);
  else column_sums_bf16<C::NT>(c, wg - ta - tb, (float*)smem);
}
template <int NT>
__global__ __launch_bounds__(NT) void sk_column_sums(ColumnSums c) {
  __shared__ float run[NT];
  column_sums_bf16<NT>(c, blockIdx.x, run);
}

// Few outputs: a workgroup takes 16 x 16 of them, and its NWK waves share out the blocks of K in turn (wave w:
// blocks w, w + NWK, ...), so that together they read whole stretches of each row of B.  The operands go
// straight to registers, U blocks at a time, with no barrier before the end, where the waves' sums are added in LDS in
// wave order.  Bound by reading B once.
template <int NWK, int U, bool BROW>
__global__ __launch_bounds__(64 * NWK) void sk_gemm_block_rows(BlockGemm g) {
  __shared__ __attribute__((aligned(16))) float red[NWK][64][4];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int lr = lane & 15, lg = lane >> 4;
  const int tn = blockIdx.x % g.tiles_n, tm = blockIdx.x / g.tiles_n;
  const int m0 = tm * 16, n0 = tn * 16;
  const int rows = min(16, g.M - m0), cols = min(16, g.N - n0);
  const uint32_t rb = (uint32_t)g.row_bytes;
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(g.A + (int64_t)m0 * rb, (uint32_t)rows * rb);
  const __amdgpu_buffer_rsrc_t rbr = make_rsrc(g.B + (int64_t)n0 * rb, (uint32_t)cols * rb);
  v4f acc = v4f{};

  for (int k0 = wave; k0 < g.kb; k0 += NWK * U) {
    v4u a[U][2], b[U][2];
    float sa[U];
    v4f sb[U];
    // all of B's first: they come from memory, A's from the caches
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = k0 + u * NWK;
        const uint32_t c = (uint32_t)(k * kBlock + 16 * lg + 64 * h);
        const bool in = k < g.kb && c < rb;
        b[u][h] = __builtin_amdgcn_raw_buffer_load_b128(rbr, in ? (uint32_t)lr * rb + c : kOob, 0, 0);
      }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * NWK;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t c = (uint32_t)(k * kBlock + 16 * lg + 64 * h);
        const bool in = k < g.kb && c < rb;
        a[u][h] = __builtin_amdgcn_raw_buffer_load_b128(ra, in ? (uint32_t)lr * rb + c : kOob, 0, 0);
      }
      const int ks = min(k, g.kb - 1);
      const float s = g.SA[(int64_t)ks * g.M + min(m0 + lr, g.M - 1)];
      sa[u] = k < g.kb ? s : 0.0f;
      if constexpr (BROW) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float sq = g.SB[(int64_t)ks * g.N + min(n0 + 4 * lg + q, g.N - 1)];
          sb[u][q] = k < g.kb ? sq : 0.0f;
        }
      } else {
        const float sq = g.SB[(int64_t)(n0 / kBlock) * g.kb + ks];
        sb[u][0] = k < g.kb ? sq : 0.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const v4f p = block_mfma(b[u], a[u]);
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[q] = __builtin_fmaf(sa[u] * sb[u][BROW ? q : 0], p[q], acc[q]);
    }
  }
  *(v4f*)red[wave][lane] = acc;
  __syncthreads();
  if (wave) return;
  v4f x = *(const v4f*)red[0][lane];
#pragma unroll
  for (int w = 1; w < NWK; ++w) x += *(const v4f*)red[w][lane];
  const int row = m0 + lr, col = n0 + 4 * lg;
  if (row >= g.M || col >= g.N) return;
  float bias[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) bias[k] = g.bias && col + k < g.N ? bits_f((uint32_t)g.bias[col + k] << 16) : 0.0f;
  const v2u h = out4(x, bias);
  uint16_t* const o = g.C + (int64_t)row * g.N + col;
  if ((g.N & 3) == 0) {
    *(v2u*)o = h;
  } else {
    const uint32_t v[4] = {h[0] & 0xffffu, h[0] >> 16, h[1] & 0xffffu, h[1] >> 16};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (col + k < g.N) o[k] = (uint16_t)v[k];
  }
}

template <class C>
hipError_t launch_tiled(BlockGemm g, bool b_tile, int grid_cap, int cus, hipStream_t s) {
  if constexpr (C::EARLY_A && !C::STREAM) {
    // Such a tile fills a compute unit, and where there are several to each, one workgroup to a unit takes every cus-th as one
    // stream: 8192x8192x512 65 -> 52 us, 8192x8192x2048 130 -> 124, 8192x8192x4096 227 -> 225, but 6144 327 / 327 and
    // 8192 424 / 430, where the units' different speeds tell (they are dealt single tiles as they become free).  With a scale
    // per row of B, whose loop has no registers to spare: 8192x8192x512 70.5 -> 59.4 us, 4096x8192x2048 81.1 / 80.8,
    // 6000x6000x4000 193.4 / 196.6.
    if (g.kb > C::STAGES && g.kb < (b_tile ? 48 : 16) && (int64_t)cdiv(g.M, C::BM) * cdiv(g.N, C::BN) > cus)
      return launch_tiled<BlockCfg<C::BM, C::BN, C::WM, C::WN, C::STAGES, 1, true>>(g, b_tile, cus, cus, s);
  }
  g.tiles_m = cdiv(g.M, C::BM);
  g.tiles_n = cdiv(g.N, C::BN);
  const int64_t T = (int64_t)g.tiles_m * g.tiles_n;
  if (T > 0x7fffffff) return hipErrorInvalidValue;
  const int grid = grid_cap > 0 && grid_cap < T ? grid_cap : (int)T;
  return launch(b_tile ? sk_gemm_block<C, false> : sk_gemm_block<C, true>, dim3(grid), C::NT, s, g);
}

template <int NWK, int U>
hipError_t launch_rows(BlockGemm g, bool b_tile, hipStream_t s) {
  g.tiles_m = cdiv(g.M, 16);
  g.tiles_n = cdiv(g.N, 16);
  return launch(b_tile ? sk_gemm_block_rows<NWK, U, false> : sk_gemm_block_rows<NWK, U, true>,
                dim3((unsigned)(g.tiles_m * g.tiles_n)), 64 * NWK, s, g);
}

template <class C>
hipError_t launch_pair(BlockGemm a, BlockGemm b, const ColumnSums& c, hipStream_t s) {
  for (BlockGemm* g : {&a, &b}) {
    g->tiles_m = g->C ? cdiv(g->M, C::BM) : 0;
    g->tiles_n = g->C ? cdiv(g->N, C::BN) : 0;
  }
  const int64_t sums = c.out ? cdiv(c.N, C::NT / kSumSlices) : 0;
  const int64_t grid = (int64_t)a.tiles_m * a.tiles_n + (int64_t)b.tiles_m * b.tiles_n + sums;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  return launch(sk_gemm_block_pair<C>, dim3((unsigned)grid), C::NT, s, a, b, c);
}

// The tile by how many of each shape there are to `cus` compute units (times below: 256 of them, one product).  A tile
// twice as large reads half as much for each product, so the largest shape that keeps most units busy is
// taken; below that, the smallest tiles that still run all at once, with waves sharing out K to shorten it.
// (kb: the product's blocks of K; rows: its rows.)
template <class Tiles, class Go>
hipError_t choose_tile(Tiles&& tiles, int rows, int kb, int cus, Go&& go) {
  // 512x512x8192 10.7 us against 14.8 with 64x32 tiles and 15.8 with 64x64
  if (rows <= 32 || tiles(32, 32) <= cus) return go(BlockCfg<32, 32, 1, 1, 3, 4>{});
  // 500x700x900 5.7 us against 6.4 with 64x64 tiles, 100x4096x4096 9.8 / 10.3
  if (rows <= 64 || tiles(64, 32) <= cus) return go(BlockCfg<64, 32, 2, 1, 3, 2>{});
  // two groups of waves pay from 16 blocks on: 128x8192x8192 28.3 -> 25.4 us, but 1024x1024x1024 6.0 -> 6.6
  if (tiles(64, 64) <= cus) return kb >= 16 ? go(BlockCfg<64, 64, 2, 2, 4, 2>{}) : go(BlockCfg<64, 64, 2, 2, 4>{});
  // 1037x1290x2064 11.7 us against 13.4 with 64x64 tiles and 14.9 with 128x128
  if (tiles(128, 64) <= cus) return go(BlockCfg<128, 64, 4, 2, 4>{});
  // Large tiles, from three quarters of the units on (3000x4100x2060, 204 tiles, 35.3 us against 46.7 with 256x128 and 47.5
  // with 128x128), or where the 128x128 ones would not run all at once and K is not short (3000x3000x8000, 144 tiles,
  // 100 us against 133 and 123; 2200x4096x2048 26.6 / 34.9 / 29.8; but 4500x2100x700 20.3 / 23.2 / 17.6).
  if (tiles(256, 256) * 4 >= (int64_t)cus * 3 || (tiles(128, 128) > 2 * (int64_t)cus && kb >= 8))
    return go(BlockCfg<256, 256, 4, 2, 2>{});
  // one to most units, with a long K: 4096x2048x4096 39.7 us against 41.7 with 128x128 tiles; 1913x2560x1792 (160 tiles)
  // 17.4 / 16.8, 2048x3147x512 11.4 / 10.8
  const int64_t halves = tiles(256, 128);
  if (halves <= cus && halves * 4 >= (int64_t)cus * 3 && kb >= 16) return go(BlockCfg<256, 128, 4, 2, 3>{});
  // more than one to a unit: two at once, on half the stages (3000x2000x1000 14.5 us against 18.1 with four stages)
  if (tiles(128, 128) > cus) return go(BlockCfg<128, 128, 4, 2, 2>{});
  // 777x4096x2048 12.5 us against 16.9 with 128x64 tiles and 19.3 with 64x64 (12.9 with the waves as 4 x 2)
  return go(BlockCfg<128, 128, 2, 4, 4>{});
}

}  // namespace

hipError_t launch_gemm_block(const BlockGemm& g, bool b_tile, int grid_cap, int cus, hipStream_t s) {
  if (grid_cap > 0 && grid_cap < cus) cus = grid_cap;
  auto tiles = [&](int bm, int bn) { return (int64_t)cdiv(g.M, bm) * cdiv(g.N, bn); };
  // Straight to registers where 16 x 16 blocks of C fill the device about once (twice, with a short K): no LDS between the
  // loads and the MFMAs, and the most waves to a block.  256x256x512 3.4 us against 4.1 with 32x32 tiles, 64x1024x1024
  // 3.4 / 4.5, 64x2048x1024 4.2 / 4.5, but 512x512x1024 (1024 blocks) 6.3 / 4.5 and 8x8192x4096 10.2 / 8.9: A is read
  // for every 16 columns instead of 32.  With a long K, 16 waves that ask for two blocks at a time:
  // 1x4096x4096 5.5 us against 6.5 with 8 and one, 256x256x2048 5.0 / 4.4.
  if (grid_cap <= 0 && tiles(16, 16) <= (g.kb <= 16 ? 2 : 1) * (int64_t)cus)
    return g.kb < 32 ? launch_rows<8, 1>(g, b_tile, s) : launch_rows<16, 2>(g, b_tile, s);
  return choose_tile(tiles, g.M, g.kb, cus, [&](auto cfg) { return launch_tiled<decltype(cfg)>(g, b_tile, grid_cap, cus, s); });
}

// Everything is chosen by both products' sizes also where only one is wanted, so that its bits are the same.
hipError_t launch_gemm_block_pair(const BlockGemm& a, const BlockGemm& b, const ColumnSums& c, int cus, hipStream_t s) {
  // One much longer along K has few outputs, so tiles that suit the other leave most units idle over its k-steps: one
  // after the other, each with tiles of its own, the sums beside the shorter.  (K of 27 blocks and 2) 3362x224x540
  // 27.6 -> 18.9 us, (32 and 3) 4096x300x4000 71 -> 39, but (13 and 3) 1652x384x1646 19.1 -> 20.7, (12 and 27)
  // 3456x1447x69 21.9 -> 24.1.
  if ((a.kb >= 16 && a.kb >= 4 * b.kb) || (b.kb >= 16 && b.kb >= 4 * a.kb)) {
    const bool a_short = a.kb < b.kb;
    const BlockGemm &first = a_short ? a : b, &second = a_short ? b : a;
    hipError_t e = hipSuccess;
    if (first.C || c.out) {
      auto tiles = [&](int bm, int bn) { return (int64_t)cdiv(first.M, bm) * cdiv(first.N, bn); };
      e = choose_tile(tiles, first.M, first.kb, cus, [&](auto cfg) {
        return launch_pair<decltype(cfg)>(a_short ? a : BlockGemm{}, a_short ? BlockGemm{} : b, c, s);
      });
    }
    return e != hipSuccess || !second.C ? e : launch_gemm_block(second, !a_short, 0, cus, s);
  }
  auto tiles = [&](int bm, int bn) {
    return (int64_t)cdiv(a.M, bm) * cdiv(a.N, bn) + (int64_t)cdiv(b.M, bm) * cdiv(b.N, bn);
  };
  const int rows = a.M > b.M ? a.M : b.M, kb = a.kb < b.kb ? a.kb : b.kb;
  return choose_tile(tiles, rows, kb, cus, [&](auto cfg) { return launch_pair<decltype(cfg)>(a, b, c, s); });
}

hipError_t launch_column_sums_bf16(const ColumnSums& c, hipStream_t s) {
  constexpr int NT = 512;
  return launch(sk_column_sums<NT>, dim3((unsigned)cdiv(c.N, NT / kSumSlices)), NT, s, c);
}

}  // namespace sk

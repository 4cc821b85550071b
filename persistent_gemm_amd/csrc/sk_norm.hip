// Root-mean-square norms before and after a block, with what stands next to them in one pass:
//
//   after a block:   out = residual_scale * residual + gate * (h rstd weight)      (h given)
//   before a block:  y = v rstd_next next_weight, v = out as stored (or x)         (next_weight given)
//                    as it is, or as E4M3 codes with a scale per 128 for the product that follows
//   rstd = (mean of squares + eps)^-1/2
//
// and their gradients.  A row is held in registers by TPR threads (a wave, with four rows to a workgroup, or
// a workgroup), CH pieces of eight elements each, so every tensor is read once and written once: all of it
// is bound by HBM (by latency for few rows).  Sums are fp32, a row's of squares across threads 64 bits.  Rows need no alignment beyond
// their elements' (a row of odd length starts anywhere).  Gated, with the next norm in fp8, 16384x4096 bf16: 103 us,
// 4.6 TB/s (a copy of 2 GiB: 4.9).  Backward of both, 4095x2047 fp32: 62 us, 3.8 TB/s, 6 us of it the column sums.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sk_common.h"
#include "sk_fp8.h"

namespace sk {

namespace {

constexpr int ceil_div(int a, int b) { return (a + b - 1) / b; }

// The sum over the TPR threads of a row, in each of them.  `red`: two areas of 16 sums, used in turn, so that
// one barrier a sum is enough (whoever writes an area again has passed the barrier after its last reading).
template <int TPR, class T>
__device__ __forceinline__ T row_sum(T x, T (*red)[16], int& turn) {
  x = wave_sum(x);
  if constexpr (TPR > 64) {
    T* const r = red[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) r[threadIdx.x >> 6] = x;
    __syncthreads();
    if constexpr (sizeof(T) == 8 || TPR == 1024) {
      // a lane for each wave's sum, the same again in every TPR / 64 lanes.  All of them in each lane take more registers:
      // doubles then spill 7 with 512 threads (gated to fp8, 2048x8000 fp32, 62.7 -> 66.8 us), floats with 1024 threads
      // more than they do (backward 2048x12000 fp32 820 -> 990 us, in bf16 685 -> 650; 2048x20000 fp32 2860 -> 3210).
      x = r[threadIdx.x & (TPR / 64 - 1)];
      if constexpr (TPR >= 1024) x += row_rotated<8>(x);
      if constexpr (TPR >= 512) x += row_rotated<4>(x);
      x += row_rotated<2>(x);
      x += row_rotated<1>(x);
    } else {
      x = r[0];
#pragma unroll
      for (int w = 1; w < TPR / 64; ++w) x += r[w];
    }
  }
  return x;
}

template <int TPR>
constexpr int rows_per_wg() { return TPR == 64 ? 4 : 1; }

// Column `col` of the row at p: p is the same in every lane and the column an unsigned 32-bit offset, which is one
// register for all of a row's tensors (instead of a 64-bit address for each).
template <class T>
__device__ __forceinline__ T* at_col(T* p, int col) { return p + (uint32_t)col; }

// The thread's row of the workgroup's, the same for a whole wave.
template <int TPR>
__device__ __forceinline__ int sub_row() { return TPR == 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x / 64) : 0; }

// One piece of eight of each of a row's CH.
template <class T, int CH>
struct RawRow {
  Raw8<T> c[CH];
};
// Row `row` of base, asked for; settle_row() where it is first used.  (base is the same in every lane, NULL for none)
template <bool SHORT, class T, int TPR, int CH>
__device__ __forceinline__ RawRow<T, CH> load_row(const void* base, int row, int t, int D) {
  RawRow<T, CH> r = {};
  if (base) {
    const T* const p = (const T*)base + (int64_t)row * D;
#pragma unroll
    for (int c = 0; c < CH; ++c) r.c[c] = load_raw8<SHORT>(p, 8 * (t + c * TPR), D);
  }
  return r;
}
template <bool SHORT, int TPR, class T, int CH>
__device__ __forceinline__ void settle_row(RawRow<T, CH>& r, int t, int D) {
#pragma unroll
  for (int c = 0; c < CH; ++c) settle8<SHORT>(r.c[c], 8 * (t + c * TPR), D);
}

// a + b of products that are rounded before: the formula's operations one by one, as a caller would write them.
__device__ __forceinline__ float sum(float a, float b) {
#pragma clang fp contract(off)
  return a + b;
}

// Has the row unpacked again where it is next used, instead of kept as floats from before: twice the registers.
template <class T, int CH>
__device__ __forceinline__ void repack(RawRow<T, CH>& r) {
  if constexpr (sizeof(T) == 2 && CH > 1) {
#pragma unroll
    for (int c = 0; c < CH; ++c) asm volatile("" : "+v"(r.c[c].w[0]));
  }
}

// ---------------------------------------------------------------- forward

// A workgroup takes consecutive rows (a wave of four: every fourth of them).  Each row's tensors are asked for one
// row ahead and kept as they lie in memory, and the vectors shared by the rows stay in registers where they
// fit (HOLD), so that the two sums of a row, which wait for all its threads, do not wait for memory.
// The scales of eight rows leave together: one row's are T apart, 4 bytes in a line each.
// Four waves to a SIMD, at most 128 registers, since the launch is for 1024 threads to a compute unit (with 129, fp32 rows of
// 512 threads ran alone on theirs: gated to fp8, 2048x8000, 62.3 -> 68.7 us).
template <class T, bool POST, bool PRE, bool FP8, int TPR, int CH, bool SHORT>
__global__ __launch_bounds__(TPR == 64 ? 256 : TPR, 4) void sk_norm_forward(NormArgs a) {
  constexpr int RPW = rows_per_wg<TPR>();
  constexpr bool HOLD = CH * sizeof(T) <= 4, AHEAD = CH < 4;   // (a wide row's registers hold little else)
  constexpr bool BATCH = FP8 && TPR > 64;
  constexpr int ROWS = 8;                       // rows whose scales leave together
  constexpr int BLOCKS = BATCH ? TPR * CH / 16 : 1;
  __shared__ double red[2][16];
  __shared__ float scales[BLOCKS][ROWS + 1];
  int turn = 0;
  const int t = threadIdx.x % TPR, D = a.D;
  // (the same in every lane, said so: two registers of the few that wide rows leave)
  const double quotient = 1.0 / (double)D;
  const double inv = __hiloint2double(__builtin_amdgcn_readfirstlane(__double2hiint(quotient)),
                                      __builtin_amdgcn_readfirstlane(__double2loint(quotient)));
  // A thread's squares, 32 at most, are summed in fp32 and the threads' sums in 64 bits: roundings do not add up with the
  // width, and a row overflows where 32 of its squares do, not where all of them would.
  auto rstd_of = [&](float squares) { return rsqrtf((float)(row_sum<TPR>((double)squares, red, turn) * inv + (double)a.eps)); };
  const int first = (int)((int64_t)a.T * blockIdx.x / gridDim.x), last = (int)((int64_t)a.T * (blockIdx.x + 1) / gridDim.x);
  typedef RawRow<T, CH> Row;
  auto load = [&](const void* p, int row) { return load_row<SHORT, T, TPR, CH>(p, row, t, D); };
  auto settle = [&](Row& r) { settle_row<SHORT, TPR>(r, t, D); };

  Row w, rs, nw;
  auto load_post = [&]() {
    w = load(a.weight, 0);
    rs = load(a.residual_scale, 0);
    settle(w);
    settle(rs);
  };
  auto load_pre = [&]() {
    nw = load(a.next_weight, 0);
    settle(nw);
  };
  if constexpr (HOLD && POST) load_post();
  if constexpr (HOLD && PRE) load_pre();
  int row = first + sub_row<TPR>();
  Row x0, h0;
  // (past the last row, the last one again)
  auto ask = [&](int r) {
    x0 = load(a.residual, min(r, last - 1));
    if constexpr (POST) h0 = load(a.h, min(r, last - 1));
  };
  if constexpr (AHEAD) ask(row);
  for (; row < last; row += RPW) {
    const int64_t at = (int64_t)row * D;
    const bool more = row + RPW < last;
    float v[CH][8];
    if constexpr (!AHEAD) ask(row);
    Row g;
    if constexpr (POST) {
      if constexpr (!HOLD) load_post();
      g = load(a.gate, row / a.gate_rows);
      settle(h0);
      float ss = 0.0f;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float h = raw_at(h0.c[c], k);
          ss = __builtin_fmaf(h, h, ss);
        }
      const float r = rstd_of(ss);
      if (t == 0) a.rstd[row] = r;
      settle(x0);
      settle(g);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = 8 * (t + c * TPR), n = min(8, max(0, D - col));
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float y = raw_at(h0.c[c], k) * r * raw_at(w.c[c], k), x = raw_at(x0.c[c], k);
          if (a.gate) y *= raw_at(g.c[c], k);
          if (a.residual_scale) x *= raw_at(rs.c[c], k);
          v[c][k] = sum(x, y);
        }
        store8(at_col((T*)a.out + at, col), n, v[c]);
        // the next norm reads what is stored
#pragma unroll
        for (int k = 0; k < 8; ++k) v[c][k] = rounded<T>(v[c][k]);
      }
    } else {
      settle(x0);
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) v[c][k] = raw_at(x0.c[c], k);
    }
    if constexpr (AHEAD) ask(row + RPW);
    if constexpr (PRE) {
      if constexpr (!HOLD) load_pre();
      float ss = 0.0f;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = __builtin_fmaf(v[c][k], v[c][k], ss);
      const float r = rstd_of(ss);
      if (t == 0) a.rstd_next[row] = r;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = 8 * (t + c * TPR), n = min(8, max(0, D - col));
#pragma unroll
        for (int k = 0; k < 8; ++k) v[c][k] = v[c][k] * r * raw_at(nw.c[c], k);
        if constexpr (FP8) {
          uint32_t m = 0;
#pragma unroll
          for (int k = 0; k < 8; ++k) m = max(m, f_bits(v[c][k]) & kAbs);
          const BlockScale b = Coder<float>::scale(max16(m));     // 16 lanes hold a block of 128
          Coder<float>::nudge(v[c], b);
          // rows hold D rounded up to 16 codes: a piece of eight is inside or outside as a whole
          if (col < a.pitch)
            *(u32x2*)at_col(a.q + (int64_t)row * a.pitch, col) = u32x2{codes4(v[c][0], v[c][1], v[c][2], v[c][3], b.s),
                                                                codes4(v[c][4], v[c][5], v[c][6], v[c][7], b.s)};
          if ((t & 15) == 0) {
            if constexpr (BATCH) scales[(t + c * TPR) / 16][row % ROWS] = b.s;
            else if (col < D) a.scale[(int64_t)(col / kBlock) * a.T + row] = b.s;
          }
        } else {
          store8(at_col((T*)a.y + at, col), n, v[c]);
        }
      }
      if constexpr (BATCH) {
        if (row % ROWS == ROWS - 1 || !more) {
          // (the next row's sums stand between this reading and the next writing)
          const int row0 = max(first, row - row % ROWS), k = t % ROWS;
          __syncthreads();
          for (int blk = t / ROWS; blk < a.blocks; blk += TPR / ROWS)
            if (row - row % ROWS + k >= row0 && row - row % ROWS + k <= row)
              a.scale[(int64_t)blk * a.T + row - row % ROWS + k] = scales[blk][k];
        }
      }
    }
  }
}

// ---------------------------------------------------------------- backward

// Workers (a workgroup, or a wave of four) take runs of consecutive rows and keep the column sums of the
// weights' gradients in registers; each run lies within the tokens that share a row of the gate.  At the end a
// workgroup's four workers are added in LDS, and a second kernel adds the workgroups' sums, both in order, so the
// results repeat bit for bit.  A row's tensors are asked for one row ahead (AHEAD), and the shared vectors kept (HOLD),
// where the registers allow it.  512 threads to a compute unit: with 1024 the sums cost more than the
// waves gain (4095x2047 fp32 63 -> 71 us), and two rows of 256 threads to a workgroup wait for each other at its
// barriers (main kernel 36 -> 40 us in bf16).
//
// part: [3][workgroups][D] (weight, next_weight, residual_scale), then of the gate [workgroups][D] where all tokens
// share a row, or [chunks][D] where a row has several chunks.
template <class T, bool POST, bool PRE, int TPR, int CH, bool SHORT>
__global__ __launch_bounds__(TPR == 64 ? 256 : TPR) void sk_norm_backward(NormGradArgs a) {
  __shared__ float red[2][16];
  constexpr int RPW = rows_per_wg<TPR>();
  __shared__ float others[RPW > 1 ? RPW - 1 : 1][RPW > 1 ? 8 * CH : 1][RPW > 1 ? TPR : 1];
  int turn = 0;
  // registers of a lane: a row's tensors as they lie in memory, the column sums, the shared vectors, and the rest
  constexpr int RAW = CH * (int)sizeof(T) * 2, ROW = RAW * (1 + 2 * POST + 2 * PRE), SUM = 8 * CH * (3 * POST + PRE);
  constexpr int VEC = RAW * (2 * POST + PRE), REST = 60 + 28 * CH, MOST = TPR == 1024 ? 128 : 256;
  constexpr bool AHEAD = 2 * ROW + SUM + VEC + REST <= MOST, HOLD = AHEAD || ROW + SUM + VEC + REST <= MOST;
  const int t = threadIdx.x % TPR, D = a.D;
  const float inv = 1.0f / (float)D;
  const int sub = sub_row<TPR>(), worker = blockIdx.x * RPW + sub, workers = gridDim.x * RPW;
  const bool gate_sums = POST && a.gate && a.gate_rows > 1, one_gate = a.groups == 1;
  const int group_rows = a.T / a.groups;
  typedef RawRow<T, CH> Row;
  auto load = [&](const void* p, int row) { return load_row<SHORT, T, TPR, CH>(p, row, t, D); };
  auto settle = [&](Row& r) { settle_row<SHORT, TPR>(r, t, D); };
  struct Rows {
    Row dout, h, res, out, dy;
    float r, rn;
  };
  const void* const res = a.residual_scale ? a.residual : nullptr;
  auto ask = [&](int row) {
    Rows x;
    x.dout = load(a.dout, row);
    if constexpr (PRE) {
      x.out = load(a.out, row);
      x.dy = load(a.dy, row);
      x.rn = a.rstd_next[row];
    }
    if constexpr (POST) {
      x.h = load(a.h, row);
      x.res = load(res, row);
      x.r = a.rstd[row];
    }
    return x;
  };
  float dw[POST ? CH : 1][8] = {}, dnw[PRE ? CH : 1][8] = {}, drs[POST ? CH : 1][8] = {}, dg[POST ? CH : 1][8] = {};
  Row w, rs, nw;
  auto load_post = [&]() {
    w = load(a.weight, 0);
    rs = load(a.residual_scale, 0);
    settle(w);
    settle(rs);
  };
  auto load_pre = [&]() {
    nw = load(a.next_weight, 0);
    settle(nw);
  };
  if constexpr (HOLD && POST) load_post();
  if constexpr (HOLD && PRE) load_pre();

  const int per = ceil_div(a.chunks, workers);
  const int chunk1 = min(a.chunks, (worker + 1) * per);
  for (int chunk = worker * per; chunk < chunk1; ++chunk) {
    const int group = chunk / a.chunks_per_gate, part = chunk - group * a.chunks_per_gate;
    const int row0 = group * group_rows + part * a.rows_per_chunk;
    const int row1 = min(row0 + a.rows_per_chunk, (group + 1) * group_rows);
    const int rows = row1 - row0, last = row1 - 1;
    Rows ahead;
    if constexpr (AHEAD) ahead = ask(row0);
    for (int i = 0; i < rows; ++i) {
      const int row = row0 + i;
      const int64_t at = (int64_t)row * D;
      Rows x;
      if constexpr (AHEAD) {
        x = ahead;
        ahead = ask(min(row + 1, last));
      } else {
        x = ask(row);
      }
      if constexpr (HOLD && POST) {
        repack(w);
        repack(rs);
      }
      if constexpr (HOLD && PRE) repack(nw);
      Row g;
      if constexpr (POST) g = load(a.gate, row / a.gate_rows);
      settle(x.dout);
      float dv[CH][8];
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) dv[c][k] = raw_at(x.dout.c[c], k);
      if constexpr (PRE) {
        if constexpr (!HOLD) load_pre();
        settle(x.out);
        settle(x.dy);
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float xh = raw_at(x.out.c[c], k) * x.rn, gy = raw_at(x.dy.c[c], k);
            dnw[c][k] = __builtin_fmaf(gy, xh, dnw[c][k]);
            s = __builtin_fmaf(gy * raw_at(nw.c[c], k), xh, s);
          }
        s = row_sum<TPR>(s, red, turn) * inv;
        repack(x.out);
        repack(x.dy);
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float xh = raw_at(x.out.c[c], k) * x.rn, gn = raw_at(x.dy.c[c], k) * raw_at(nw.c[c], k);
            dv[c][k] = __builtin_fmaf(x.rn, __builtin_fmaf(-s, xh, gn), dv[c][k]);
          }
      }
      if constexpr (POST) {
        if constexpr (!HOLD) load_post();
        settle(x.h);
        settle(x.res);
        settle(g);
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int col = 8 * (t + c * TPR), n = min(8, max(0, D - col));
          float y[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            drs[c][k] = __builtin_fmaf(dv[c][k], raw_at(x.res.c[c], k), drs[c][k]);
            y[k] = a.residual_scale ? dv[c][k] * raw_at(rs.c[c], k) : dv[c][k];
          }
          store8(at_col((T*)a.dresidual + at, col), n, y);
          if (a.gate) {
            if (gate_sums) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                dg[c][k] = __builtin_fmaf(dv[c][k] * (raw_at(x.h.c[c], k) * x.r), raw_at(w.c[c], k), dg[c][k]);
            } else {
#pragma unroll
              for (int k = 0; k < 8; ++k) y[k] = dv[c][k] * (raw_at(x.h.c[c], k) * x.r) * raw_at(w.c[c], k);
              store8(at_col((T*)a.dgate + at, col), n, y);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) dv[c][k] *= raw_at(g.c[c], k);
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float hh = raw_at(x.h.c[c], k) * x.r;
            dw[c][k] = __builtin_fmaf(dv[c][k], hh, dw[c][k]);
            dv[c][k] *= raw_at(w.c[c], k);
            s = __builtin_fmaf(dv[c][k], hh, s);
          }
        }
        s = row_sum<TPR>(s, red, turn) * inv;
        repack(x.h);
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            dv[c][k] = x.r * __builtin_fmaf(-s, raw_at(x.h.c[c], k) * x.r, dv[c][k]);
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = 8 * (t + c * TPR);
        store8(at_col((T*)a.dx + at, col), min(8, max(0, D - col)), dv[c]);
      }
    }
    if constexpr (POST) {
      if (gate_sums && !one_gate) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int col = 8 * (t + c * TPR), n = min(8, max(0, D - col));
          if (a.chunks_per_gate == 1) store8((T*)a.dgate + (int64_t)group * D + col, n, dg[c]);
          else store8(a.part + ((int64_t)3 * gridDim.x + chunk) * D + col, n, dg[c]);
#pragma unroll
          for (int k = 0; k < 8; ++k) dg[c][k] = 0.0f;
        }
      }
    }
  }
  // the workgroup's workers, added in order by the first
  auto total = [&](float (*v)[8], int slot) {
    if constexpr (RPW > 1) {
      __syncthreads();
      if (sub > 0) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int k = 0; k < 8; ++k) others[sub - 1][8 * c + k][t] = v[c][k];
      }
      __syncthreads();
      if (sub > 0) return;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int o = 0; o < RPW - 1; ++o) v[c][k] += others[o][8 * c + k][t];
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = 8 * (t + c * TPR);
      store8(a.part + ((int64_t)slot * gridDim.x + blockIdx.x) * D + col, min(8, max(0, D - col)), v[c]);
    }
  };
  if constexpr (POST) {
    total(dw, 0);
    if (a.residual_scale) total(drs, 2);
    if (gate_sums && one_gate) total(dg, 3);
  }
  if constexpr (PRE) total(dnw, 1);
}

// out[d] = the sum of `count` rows of part, in a fixed order: thread (column, slice) of 32 x 32 adds the slice's
// run of rows in turn, then the runs are added in turn.
constexpr int kSlices = 32;
template <class T>
__device__ __forceinline__ void column_sum(const float* __restrict__ part, T* __restrict__ out, int count, int D,
                                           int block) {
  __shared__ float run[kSlices][32];
  const int col = threadIdx.x & 31, slice = threadIdx.x >> 5, d = block * 32 + col;
  const int per = ceil_div(count, kSlices), c0 = slice * per, c1 = min(count, c0 + per);
  float s = 0.0f;
  if (d < D) {
#pragma unroll 8
    for (int c = c0; c < c1; ++c) s += part[(int64_t)c * D + d];
  }
  run[slice][col] = s;
  __syncthreads();
  if (slice || d >= D) return;
  float x = run[0][col];
#pragma unroll
  for (int k = 1; k < kSlices; ++k) x += run[k][col];
  if constexpr (sizeof(T) == 2) out[d] = (T)pack_bf16(x, x);
  else out[d] = x;
}

// The norms' sums: blockIdx.y 0, 1, 2 the three vectors, then the rows of the gate.
template <class T>
__global__ __launch_bounds__(32 * kSlices) void sk_norm_sums(NormGradArgs a, int wgs) {
  const int y = blockIdx.y;
  if (y < 3) {
    T* const out = (T*)(y == 0 ? a.dweight : y == 1 ? a.dnext_weight : a.dresidual_scale);
    if (out) column_sum<T>(a.part + (int64_t)y * wgs * a.D, out, wgs, a.D, blockIdx.x);
  } else {
    const int group = y - 3;
    column_sum<T>(a.part + ((int64_t)3 * wgs + (int64_t)group * a.chunks_per_gate) * a.D,
                  (T*)a.dgate + (int64_t)group * a.D, a.groups == 1 ? wgs : a.chunks_per_gate, a.D, blockIdx.x);
  }
}

template <class T, bool POST, bool PRE, bool FP8, int TPR, int CH, bool SHORT = false>
hipError_t forward(const NormArgs& a, int cus, hipStream_t s) {
  const int rpw = rows_per_wg<TPR>(), threads = TPR == 64 ? 256 : TPR;
  // as many workgroups as run at once (about 1024 threads to a compute unit), each on a run of rows
  const int wgs = ceil_div(a.T, rpw), most = cus * (1024 / threads);
  return launch(sk_norm_forward<T, POST, PRE, FP8, TPR, CH, SHORT>, dim3(min(wgs, most)), threads, s, a);
}

template <class T, bool POST, bool PRE, bool FP8>
hipError_t forward_width(const NormArgs& a, int cus, hipStream_t s) {
  if (a.D < 8) return forward<T, POST, PRE, FP8, 64, 1, true>(a, cus, s);
  // Few rows: more threads to each, to shorten the call.  Many: as few as hold the row.
  if (a.T <= 2 * cus && a.D > 512) {
    if (a.D <= 2048) return forward<T, POST, PRE, FP8, 256, 1>(a, cus, s);
    if (a.D <= 8192) return forward<T, POST, PRE, FP8, 1024, 1>(a, cus, s);
  }
  if (a.D <= 512) return forward<T, POST, PRE, FP8, 64, 1>(a, cus, s);
  if (a.D <= 1024) return forward<T, POST, PRE, FP8, 64, 2>(a, cus, s);
  if (a.D <= 2048) return forward<T, POST, PRE, FP8, 256, 1>(a, cus, s);
  if (a.D <= 4096) return forward<T, POST, PRE, FP8, 256, 2>(a, cus, s);
  if (a.D <= 8192) return forward<T, POST, PRE, FP8, 512, 2>(a, cus, s);
  if (a.D <= 16384) return forward<T, POST, PRE, FP8, 1024, 2>(a, cus, s);
  return forward<T, POST, PRE, FP8, 1024, 4>(a, cus, s);
}

template <class T>
hipError_t forward_form(const NormArgs& a, int cus, hipStream_t s) {
  if (!a.h) return a.q ? forward_width<T, false, true, true>(a, cus, s) : forward_width<T, false, true, false>(a, cus, s);
  if (!a.next_weight) return forward_width<T, true, false, false>(a, cus, s);
  return a.q ? forward_width<T, true, true, true>(a, cus, s) : forward_width<T, true, true, false>(a, cus, s);
}

// Threads of a row in the backward, and workers of a workgroup.
int grad_threads(int D) { return D <= 512 ? 64 : D <= 2048 ? 256 : D <= 8192 ? 512 : 1024; }
int grad_rpw(int D) { return D <= 512 ? 4 : 1; }
// No more workers than run at once, each with its share of the chunks (as many as there are rows of the gate, perhaps): every
// workgroup writes rows of sums, D long.  8192x4096 bf16 with 4096 rows of the gate 203 -> 121 us, its scratch 201 -> 13 MB.
int grad_wgs(const NormGradArgs& a) { return ceil_div(a.chunks, grad_rpw(a.D) * ceil_div(a.chunks, a.workers)); }

template <class T, bool POST, bool PRE, int TPR, int CH, bool SHORT = false>
hipError_t backward(const NormGradArgs& a, hipStream_t s) {
  const int wgs = grad_wgs(a);
  const hipError_t e = launch(sk_norm_backward<T, POST, PRE, TPR, CH, SHORT>, dim3(wgs), TPR == 64 ? 256 : TPR, s, a);
  if (e != hipSuccess) return e;
  const bool gate = a.dgate && a.gate_rows > 1 && (a.groups == 1 || a.chunks_per_gate > 1);
  return launch(sk_norm_sums<T>, dim3(ceil_div(a.D, 32), 3 + (gate ? a.groups : 0)), 32 * kSlices, s, a, wgs);
}

template <class T, bool POST, bool PRE>
hipError_t backward_width(const NormGradArgs& a, hipStream_t s) {
  if (a.D < 8) return backward<T, POST, PRE, 64, 1, true>(a, s);
  switch (grad_threads(a.D)) {
    case 64: return backward<T, POST, PRE, 64, 1>(a, s);
    case 256: return backward<T, POST, PRE, 256, 1>(a, s);
    case 512: return a.D <= 4096 ? backward<T, POST, PRE, 512, 1>(a, s) : backward<T, POST, PRE, 512, 2>(a, s);
    default: return a.D <= 16384 ? backward<T, POST, PRE, 1024, 2>(a, s) : backward<T, POST, PRE, 1024, 4>(a, s);
  }
}

template <class T>
hipError_t backward_form(const NormGradArgs& a, hipStream_t s) {
  if (!a.h) return backward_width<T, false, true>(a, s);
  return a.dy ? backward_width<T, true, true>(a, s) : backward_width<T, true, false>(a, s);
}

}  // namespace

hipError_t launch_norm_forward(const NormArgs& a, bool f32, int cus, hipStream_t s) {
  if (a.D > kMaxNormWidth) return hipErrorInvalidValue;
  return f32 ? forward_form<float>(a, cus, s) : forward_form<uint16_t>(a, cus, s);
}

// Sets the partition of the rows and returns the bytes of `part`.
int64_t norm_grad_scratch_bytes(NormGradArgs* a, int cus) {
  const bool grouped = a->h && a->gate && a->gate_rows > 1;
  a->groups = grouped ? a->T / a->gate_rows : 1;
  const int group_rows = a->T / a->groups;
  // 512 threads to a compute unit (a stream may be held to one, which has to take a row of 1024)
  const int want = a->workers = max(1, 512 * cus / grad_threads(a->D));
  a->chunks_per_gate = a->groups >= want ? 1 : ceil_div(want, a->groups);
  a->rows_per_chunk = ceil_div(group_rows, a->chunks_per_gate);
  a->chunks_per_gate = ceil_div(group_rows, a->rows_per_chunk);
  a->chunks = a->groups * a->chunks_per_gate;
  const int64_t wgs = grad_wgs(*a), gate = !grouped ? 0 : a->groups == 1 ? wgs : a->chunks_per_gate > 1 ? a->chunks : 0;
  return (3 * wgs + gate) * (int64_t)a->D * (int64_t)sizeof(float);
}

hipError_t launch_norm_backward(const NormGradArgs& a, bool f32, hipStream_t s) {
  if (a.D > kMaxNormWidth) return hipErrorInvalidValue;
  return f32 ? backward_form<float>(a, s) : backward_form<uint16_t>(a, s);
}

}  // namespace sk

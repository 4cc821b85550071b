// C ABI of the block-scaled E4M3 operators and the norms around them: argument checks and launches.

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>

#include "../../include/sk_gemm.h"
#include "sk_common.h"
#include "sk_host.h"

namespace {

using sk::host::overlaps;

constexpr int64_t kMaxRows = ((int64_t)1 << 31) - (1 << 20);   // (row indices step past the end in 32 bits)

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t up(int64_t a, int64_t b) { return cdiv(a, b) * b; }
bool misaligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) != 0; }

// One range of memory of a call.
struct Range {
  const void* p;
  int64_t n;
};

// Whether an output shares bytes with an input or with another output.
bool clash(const Range* in, int n_in, const Range* out, int n_out) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlaps(out[i].p, out[i].n, in[j].p, in[j].n)) return true;
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n)) return true;
  }
  return false;
}

bool elem_ok(int e) { return e == SK_ELEM_BF16 || e == SK_ELEM_F32; }
bool block_ok(int b) { return b == SK_BLOCK_ROW || b == SK_BLOCK_TILE; }
int64_t elem_size(int e) { return e == SK_ELEM_F32 ? 4 : 2; }

// One product (checked arguments).
sk::BlockGemm product(const void* A, const void* B, const float* sa, const float* sb, const void* bias, void* C,
                      int64_t M, int64_t N, int64_t K) {
  sk::BlockGemm g;
  std::memset(&g, 0, sizeof(g));
  g.A = (const uint8_t*)A;
  g.B = (const uint8_t*)B;
  g.SA = sa;
  g.SB = sb;
  g.bias = (const uint16_t*)bias;
  g.C = (uint16_t*)C;
  g.M = (int)M;
  g.N = (int)N;
  g.row_bytes = (int)K;
  g.kb = (int)cdiv(K, 128);
  return g;
}

sk_status ok(hipError_t e) { return e == hipSuccess ? SK_OK : SK_ERR_HIP; }

}  // namespace

extern "C" {

sk_status sk_quantize_fp8_block(const void* x, sk_elem elem, sk_block block, void* q, float* scale, void* qt,
                                float* scale_t, int64_t R, int64_t C, void* stream) {
  if (!elem_ok(elem) || !block_ok(block) || !x) return SK_ERR_ARG;
  if (!q != !scale || !qt != !scale_t || (!q && !qt)) return SK_ERR_ARG;
  if (R < 1 || C < 1 || R >= kMaxRows || C >= kMaxRows) return SK_ERR_ARG;
  const int64_t kb = cdiv(C, 128), rb = cdiv(R, 128);
  if (kb * rb >= (int64_t)1 << 31) return SK_ERR_ARG;
  const int64_t e = elem_size(elem);
  if (misaligned(x, (uintptr_t)e) || misaligned(q, 16) || misaligned(qt, 16) || misaligned(scale, 4) ||
      misaligned(scale_t, 4))
    return SK_ERR_ALIGN;
  const bool tile = block == SK_BLOCK_TILE;
  const Range in[] = {{x, R * C * e}};
  const Range out[] = {{q, R * up(C, 16)},
                       {scale, 4 * kb * (tile ? rb : R)},
                       {qt, C * up(R, 16)},
                       {scale_t, 4 * rb * (tile ? kb : C)}};
  if (clash(in, 1, out, 4)) return SK_ERR_ARG;
  int dev = 0, cus = 0;
  sk_status st = sk::host::device_for((hipStream_t)stream, &dev, &cus);
  if (st != SK_OK) return st;
  sk::QuantArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = x;
  a.q = (uint8_t*)q;
  a.scale = scale;
  a.qt = (uint8_t*)qt;
  a.scale_t = scale_t;
  a.R = (int)R;
  a.C = (int)C;
  a.pitch = (int)up(C, 16);
  a.pitch_t = (int)up(R, 16);
  a.kb = (int)kb;
  a.rb = (int)rb;
  return sk::launch_quantize_block(a, elem == SK_ELEM_F32, tile, (hipStream_t)stream) == hipSuccess ? SK_OK : SK_ERR_HIP;
}

sk_status sk_gemm_fp8_block(const void* A, const void* B, const float* A_scale, const float* B_scale, sk_block b_block,
                            const void* bias, void* C, int64_t M, int64_t N, int64_t K, int grid_cap, void* stream) {
  if (!A || !B || !A_scale || !B_scale || !C || !block_ok(b_block)) return SK_ERR_ARG;
  if (M < 1 || N < 1 || K < 1 || M >= kMaxRows || N > sk::kMaxN || K > sk::kMaxK) return SK_ERR_ARG;
  if (K % 16 || misaligned(A, 16) || misaligned(B, 16) || misaligned(C, 16) || misaligned(A_scale, 4) ||
      misaligned(B_scale, 4) || misaligned(bias, 2))
    return SK_ERR_ALIGN;
  const bool tile = b_block == SK_BLOCK_TILE;
  const int64_t kb = cdiv(K, 128);
  if (cdiv(M, 16) * cdiv(N, 16) >= (int64_t)1 << 31) return SK_ERR_ARG;
  const Range in[] = {{A, M * K}, {B, N * K}, {A_scale, 4 * kb * M}, {B_scale, 4 * kb * (tile ? cdiv(N, 128) : N)},
                      {bias, 2 * N}};
  const Range out[] = {{C, 2 * M * N}};
  if (clash(in, 5, out, 1)) return SK_ERR_ARG;
  int dev = 0, cus = 0;
  sk_status st = sk::host::device_for((hipStream_t)stream, &dev, &cus);
  if (st != SK_OK) return st;
  return ok(sk::launch_gemm_block(product(A, B, A_scale, B_scale, bias, C, M, N, K), tile, grid_cap, cus,
                                  (hipStream_t)stream));
}

sk_status sk_gemm_fp8_block_backward(const void* dC, const void* At, const float* At_scale, const void* Bt,
                                     const float* Bt_scale, void* dA, void* dB, void* dbias, int64_t M, int64_t N,
                                     int64_t K, int grid_cap, void* stream) {
  if (!dC || (!dA && !dB && !dbias)) return SK_ERR_ARG;
  if ((dA && (!Bt || !Bt_scale)) || (dB && (!At || !At_scale))) return SK_ERR_ARG;
  // dA sums over N (its operand rows are N codes long), dB over M; K is an output width
  if (M < 1 || N < 1 || K < 1 || M >= kMaxRows || N >= kMaxRows || K > sk::kMaxN) return SK_ERR_ARG;
  if ((dA && N > sk::kMaxK) || (dB && M > sk::kMaxK)) return SK_ERR_ARG;
  const int64_t mb = cdiv(M, 128), nb = cdiv(N, 128), kb = cdiv(K, 128), mp = up(M, 16), np = up(N, 16);
  if (mb * nb >= (int64_t)1 << 31 || cdiv(M, 16) * cdiv(K, 16) >= (int64_t)1 << 31 ||
      cdiv(N, 16) * cdiv(K, 16) >= (int64_t)1 << 31)
    return SK_ERR_ARG;
  if (misaligned(dC, 2) || misaligned(At, 16) || misaligned(Bt, 16) || misaligned(dA, 16) || misaligned(dB, 16) ||
      misaligned(dbias, 2) || misaligned(At_scale, 4) || misaligned(Bt_scale, 4))
    return SK_ERR_ALIGN;
  const Range in[] = {{dC, 2 * M * N}, {At, K * mp}, {At_scale, 4 * mb * K}, {Bt, K * np}, {Bt_scale, 4 * kb * nb}};
  const Range out[] = {{dA, 2 * M * K}, {dB, 2 * N * K}, {dbias, 2 * N}};
  if (clash(in, 5, out, 3)) return SK_ERR_ARG;
  hipStream_t s = (hipStream_t)stream;
  sk_status st = sk::host::refuse_capture(s);
  if (st != SK_OK) return st;
  int dev = 0, cus = 0;
  st = sk::host::device_for(s, &dev, &cus);
  if (st != SK_OK) return st;
  // scratch: the codes and scales of dC and of dC^T, and the column sums of each 128 rows
  const int64_t at_s = up(dA ? M * np : 0, 256), at_qt = at_s + up(dA ? 4 * nb * M : 0, 256);
  const int64_t at_st = at_qt + up(dB ? N * mp : 0, 256), at_part = at_st + up(dB ? 4 * mb * N : 0, 256);
  uint8_t* w = nullptr;
  sk::host::Hold hold;
  st = sk::host::scratch(dev, s, (size_t)(at_part + (dbias ? 4 * mb * N : 0)), &hold, &w);
  if (st != SK_OK) return st;
  sk::QuantArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = dC;
  if (dA) {
    a.q = w;
    a.scale = (float*)(w + at_s);
  }
  if (dB) {
    a.qt = w + at_qt;
    a.scale_t = (float*)(w + at_st);
  }
  if (dbias) a.part = (float*)(w + at_part);
  a.R = (int)M;
  a.C = (int)N;
  a.pitch = (int)np;
  a.pitch_t = (int)mp;
  a.kb = (int)nb;
  a.rb = (int)mb;
  if (sk::launch_quantize_block(a, false, false, s) != hipSuccess) return SK_ERR_HIP;
  const sk::ColumnSums sums{a.part, (uint16_t*)dbias, (int)mb, (int)N};
  const sk::BlockGemm ga = product(a.q, Bt, a.scale, Bt_scale, nullptr, dA, M, K, np);
  const sk::BlockGemm gb = product(a.qt, At, a.scale_t, At_scale, nullptr, dB, N, K, mp);
  if ((dA || dB) && grid_cap <= 0) return ok(sk::launch_gemm_block_pair(ga, gb, sums, cus, s));
  if (dA && sk::launch_gemm_block(ga, true, grid_cap, cus, s) != hipSuccess) return SK_ERR_HIP;
  if (dB && sk::launch_gemm_block(gb, false, grid_cap, cus, s) != hipSuccess) return SK_ERR_HIP;
  return dbias ? ok(sk::launch_column_sums_bf16(sums, s)) : SK_OK;
}

sk_status sk_norm_forward(const sk_norm_args* p) {
  if (!p) return SK_ERR_ARG;
  const sk_norm_args& g = *p;
  if (!elem_ok(g.elem) || !g.residual || (!g.h && !g.next_weight)) return SK_ERR_ARG;
  if (g.h ? !g.weight || !g.out || !g.rstd : g.weight || g.out || g.rstd || g.gate || g.residual_scale) return SK_ERR_ARG;
  if (g.next_weight ? !g.rstd_next || !g.y == !g.q || !g.q != !g.scale : g.y || g.q || g.scale || g.rstd_next)
    return SK_ERR_ARG;
  if (g.T < 1 || g.D < 1 || g.T >= kMaxRows || g.D > sk::kMaxNormWidth) return SK_ERR_ARG;
  if (g.gate ? g.gates < 1 || g.gates > g.T || g.T % g.gates : g.gates != 0) return SK_ERR_ARG;
  const int64_t e = elem_size(g.elem), row = g.D * e, all = g.T * row, blocks = cdiv(g.D, 128);
  for (const void* v : {g.h, g.residual, g.weight, g.gate, g.residual_scale, g.next_weight, (const void*)g.out,
                        (const void*)g.y})
    if (misaligned(v, (uintptr_t)e)) return SK_ERR_ALIGN;
  if (misaligned(g.rstd, 4) || misaligned(g.rstd_next, 4) || misaligned(g.scale, 4) || misaligned(g.q, 16))
    return SK_ERR_ALIGN;
  // a row is read whole before it is written, so out may be h or residual itself
  const Range in[] = {{g.out == g.h ? nullptr : g.h, all}, {g.out == g.residual ? nullptr : g.residual, all},
                      {g.weight, row}, {g.gate, g.gates * row}, {g.residual_scale, row}, {g.next_weight, row}};
  const Range out[] = {{g.out, all}, {g.rstd, 4 * g.T}, {g.y, all}, {g.q, g.T * up(g.D, 16)},
                       {g.scale, 4 * blocks * g.T}, {g.rstd_next, 4 * g.T}};
  if (clash(in, 6, out, 6)) return SK_ERR_ARG;
  int dev = 0, cus = 0;
  sk_status st = sk::host::device_for((hipStream_t)g.stream, &dev, &cus);
  if (st != SK_OK) return st;
  sk::NormArgs a;
  std::memset(&a, 0, sizeof(a));
  a.h = g.h;
  a.residual = g.residual;
  a.weight = g.weight;
  a.gate = g.gate;
  a.residual_scale = g.residual_scale;
  a.next_weight = g.next_weight;
  a.out = g.out;
  a.rstd = g.rstd;
  a.y = g.y;
  a.q = (uint8_t*)g.q;
  a.scale = g.scale;
  a.rstd_next = g.rstd_next;
  a.eps = g.eps;
  a.T = (int)g.T;
  a.D = (int)g.D;
  a.gate_rows = g.gate ? (int)(g.T / g.gates) : 1;
  a.pitch = (int)up(g.D, 16);
  a.blocks = (int)blocks;
  return sk::launch_norm_forward(a, g.elem == SK_ELEM_F32, cus, (hipStream_t)g.stream) == hipSuccess ? SK_OK : SK_ERR_HIP;
}

sk_status sk_norm_backward(const sk_norm_grad_args* p) {
  if (!p) return SK_ERR_ARG;
  const sk_norm_grad_args& g = *p;
  if (!elem_ok(g.elem) || !g.dx || (!g.h && !g.dy)) return SK_ERR_ARG;
  if (g.dy ? !g.out || !g.next_weight || !g.rstd_next || !g.dnext_weight
           : g.out || g.next_weight || g.rstd_next || g.dnext_weight)
    return SK_ERR_ARG;
  if (g.h) {
    if (!g.dout || !g.weight || !g.rstd || !g.dresidual || !g.dweight) return SK_ERR_ARG;
    if (!g.gate != !g.dgate || !g.residual_scale != !g.dresidual_scale || (g.residual_scale && !g.residual))
      return SK_ERR_ARG;
  } else if (g.weight || g.rstd || g.gate || g.residual_scale || g.dresidual || g.dweight || g.dgate ||
             g.dresidual_scale) {
    return SK_ERR_ARG;
  }
  if (g.T < 1 || g.D < 1 || g.T >= kMaxRows || g.D > sk::kMaxNormWidth) return SK_ERR_ARG;
  if (g.gate ? g.gates < 1 || g.gates > g.T || g.T % g.gates : g.gates != 0) return SK_ERR_ARG;
  const int64_t e = elem_size(g.elem), row = g.D * e, all = g.T * row;
  for (const void* v : {g.dout, g.dy, g.out, g.next_weight, g.h, g.residual, g.weight, g.gate, g.residual_scale,
                        (const void*)g.dx, (const void*)g.dresidual, (const void*)g.dweight, (const void*)g.dgate,
                        (const void*)g.dresidual_scale, (const void*)g.dnext_weight})
    if (misaligned(v, (uintptr_t)e)) return SK_ERR_ALIGN;
  if (misaligned(g.rstd, 4) || misaligned(g.rstd_next, 4)) return SK_ERR_ALIGN;
  const Range in[] = {{g.dout, all}, {g.dy, all}, {g.out, all}, {g.next_weight, row}, {g.rstd_next, 4 * g.T},
                      {g.h, all}, {g.residual_scale ? g.residual : nullptr, all}, {g.weight, row},
                      {g.gate, g.gates * row}, {g.residual_scale, row}, {g.rstd, 4 * g.T}};
  const Range out[] = {{g.dx, all}, {g.dresidual, all}, {g.dweight, row}, {g.dgate, g.gates * row},
                       {g.dresidual_scale, row}, {g.dnext_weight, row}};
  if (clash(in, 11, out, 6)) return SK_ERR_ARG;
  hipStream_t s = (hipStream_t)g.stream;
  sk_status st = sk::host::refuse_capture(s);
  if (st != SK_OK) return st;
  int dev = 0, cus = 0;
  st = sk::host::device_for(s, &dev, &cus);
  if (st != SK_OK) return st;
  sk::NormGradArgs a;
  std::memset(&a, 0, sizeof(a));
  a.dout = g.dout;
  a.dy = g.dy;
  a.out = g.out;
  a.next_weight = g.next_weight;
  a.rstd_next = g.rstd_next;
  a.h = g.h;
  a.residual = g.residual;
  a.weight = g.weight;
  a.gate = g.gate;
  a.residual_scale = g.residual_scale;
  a.rstd = g.rstd;
  a.dx = g.dx;
  a.dresidual = g.dresidual;
  a.dweight = g.dweight;
  a.dgate = g.dgate;
  a.dresidual_scale = g.dresidual_scale;
  a.dnext_weight = g.dnext_weight;
  a.T = (int)g.T;
  a.D = (int)g.D;
  a.gate_rows = g.gate ? (int)(g.T / g.gates) : 1;
  uint8_t* w = nullptr;
  sk::host::Hold hold;
  st = sk::host::scratch(dev, s, (size_t)sk::norm_grad_scratch_bytes(&a, cus), &hold, &w);
  if (st != SK_OK) return st;
  a.part = (float*)w;
  return sk::launch_norm_backward(a, g.elem == SK_ELEM_F32, s) == hipSuccess ? SK_OK : SK_ERR_HIP;
}

}  // extern "C"

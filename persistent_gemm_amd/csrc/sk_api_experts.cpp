// C ABI of a layer of experts: routing, products grouped by expert, products with 4-bit weights.  Argument checks and
// launches.

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "../../include/sk_gemm.h"
#include "sk_common.h"
#include "sk_host.h"

namespace {

using sk::host::overlaps;

constexpr int64_t kMaxRows = ((int64_t)1 << 31) - (1 << 20);   // (row indices step past the end in 32 bits)

// Bytes of an A whose rows are chosen: lanes address it by 32-bit offsets, and those out of its range lie 2 GiB and up to a few
// k-steps above the others.
constexpr int64_t kMaxGathered = ((int64_t)1 << 31) - 4096;

bool misaligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) != 0; }
bool elem_ok(int e) { return e == SK_ELEM_BF16 || e == SK_ELEM_F16 || e == SK_ELEM_F32; }
bool half_ok(int e) { return e == SK_ELEM_BF16 || e == SK_ELEM_F16; }
int64_t size_of(int e) { return e == SK_ELEM_F32 ? 4 : 2; }
bool within(int64_t n, int64_t most) { return n >= 1 && n <= most; }

struct Range {
  const void* p;
  int64_t n;
};
// Whether an output shares bytes with an input or with another output.
bool clash(std::initializer_list<Range> in, std::initializer_list<Range> out) {
  for (const Range* o = out.begin(); o != out.end(); ++o) {
    for (const Range& i : in)
      if (overlaps(o->p, o->n, i.p, i.n)) return true;
    for (const Range* b = out.begin(); b != o; ++b)
      if (overlaps(o->p, o->n, b->p, b->n)) return true;
  }
  return false;
}

sk_status ok(hipError_t e) { return e == hipSuccess ? SK_OK : SK_ERR_HIP; }

bool route_sizes_ok(int64_t T, int64_t E, int64_t k) {
  return within(T, kMaxRows) && within(E, sk::kMaxExperts) && within(k, sk::kMaxChoices) && k <= E && T * k < kMaxRows;
}

}  // namespace

extern "C" {

int64_t sk_moe_route_work_bytes(int64_t T, int64_t E) {
  return within(T, kMaxRows) && within(E, sk::kMaxExperts) ? sk::route_blocks(T, (int)E) * E * 4 : 0;
}

sk_status sk_moe_route(const void* logits, sk_elem elem, int normalize, int32_t* experts, float* weights,
                       int32_t* offsets, int32_t* slots, int32_t* rows, void* work, int64_t T, int64_t E, int64_t k,
                       void* stream) {
  if (!elem_ok(elem) || !logits || !experts || !weights || !offsets || !slots || !rows) return SK_ERR_ARG;
  if (!route_sizes_ok(T, E, k) || (!work && sk_moe_route_work_bytes(T, E))) return SK_ERR_ARG;
  if (misaligned(logits, (uintptr_t)size_of(elem))) return SK_ERR_ALIGN;
  for (const void* p : {(const void*)experts, (const void*)weights, (const void*)offsets, (const void*)slots,
                        (const void*)rows, (const void*)work})
    if (misaligned(p, 4)) return SK_ERR_ALIGN;
  const int64_t n = 4 * T * k;
  if (clash({{logits, T * E * size_of(elem)}}, {{experts, n}, {weights, n}, {offsets, 4 * (E + 1)}, {slots, n}, {rows, n},
                                                {work, sk_moe_route_work_bytes(T, E)}}))
    return SK_ERR_ARG;
  int dev = 0, cus = 0;
  const sk_status st = sk::host::device_for((hipStream_t)stream, &dev, &cus);
  if (st != SK_OK) return st;
  sk::RouteArgs a;
  std::memset(&a, 0, sizeof(a));
  a.logits = logits;
  a.experts = experts;
  a.weights = weights;
  a.offsets = offsets;
  a.slots = slots;
  a.rows = rows;
  a.part = (int*)work;
  a.T = T;
  a.E = (int)E;
  a.k = (int)k;
  a.normalize = normalize != 0;
  return ok(sk::launch_route(a, elem, (hipStream_t)stream));
}

sk_status sk_moe_route_backward(const float* dweights, const void* logits, sk_elem elem, int normalize,
                                const int32_t* experts, const float* weights, void* dlogits, int64_t T, int64_t E,
                                int64_t k, void* stream) {
  if (!elem_ok(elem) || !dweights || !experts || !weights || !dlogits || (!normalize && !logits)) return SK_ERR_ARG;
  if (!route_sizes_ok(T, E, k)) return SK_ERR_ARG;
  if (misaligned(logits, (uintptr_t)size_of(elem)) || misaligned(dlogits, (uintptr_t)size_of(elem)) ||
      misaligned(dweights, 4) || misaligned(experts, 4) || misaligned(weights, 4))
    return SK_ERR_ALIGN;
  const int64_t n = 4 * T * k, all = T * E * size_of(elem);
  if (clash({{normalize ? nullptr : logits, all}, {dweights, n}, {experts, n}, {weights, n}}, {{dlogits, all}}))
    return SK_ERR_ARG;
  int dev = 0, cus = 0;
  const sk_status st = sk::host::device_for((hipStream_t)stream, &dev, &cus);
  if (st != SK_OK) return st;
  sk::RouteGradArgs a;
  std::memset(&a, 0, sizeof(a));
  a.dweights = dweights;
  a.logits = logits;
  a.experts = experts;
  a.weights = weights;
  a.dlogits = dlogits;
  a.T = T;
  a.E = (int)E;
  a.k = (int)k;
  a.normalize = normalize != 0;
  return ok(sk::launch_route_gradient(a, elem, (hipStream_t)stream));
}

sk_status sk_moe_combine(const void* y, sk_elem elem, const int32_t* slots, const float* weights, void* out, int64_t T,
                         int64_t k, int64_t R, int64_t D, void* stream) {
  if (!elem_ok(elem) || !y || !slots || !out) return SK_ERR_ARG;
  if (!within(T, kMaxRows) || !within(k, sk::kMaxChoices) || !within(R, kMaxRows) || !within(D, sk::kMaxN)) return SK_ERR_ARG;
  const int64_t e = size_of(elem);
  if (misaligned(y, (uintptr_t)e) || misaligned(out, (uintptr_t)e) || misaligned(slots, 4) || misaligned(weights, 4))
    return SK_ERR_ALIGN;
  if (clash({{y, R * D * e}, {slots, 4 * T * k}, {weights, 4 * T * k}}, {{out, T * D * e}})) return SK_ERR_ARG;
  int dev = 0, cus = 0;
  const sk_status st = sk::host::device_for((hipStream_t)stream, &dev, &cus);
  if (st != SK_OK) return st;
  sk::CombineArgs a;
  std::memset(&a, 0, sizeof(a));
  a.y = y;
  a.slots = slots;
  a.weights = weights;
  a.out = out;
  a.T = T;
  a.R = (int)R;
  a.D = (int)D;
  a.k = (int)k;
  return ok(sk::launch_combine(a, elem, (hipStream_t)stream));
}

sk_status sk_moe_combine_backward(const void* dout, const void* y, sk_elem elem, const int32_t* slots,
                                  const float* weights, const int32_t* offsets, void* dy, float* dweights, int64_t T,
                                  int64_t k, int64_t R, int64_t D, int64_t E, void* stream) {
  if (!elem_ok(elem) || !dout || !slots || !dy || (dweights && !y)) return SK_ERR_ARG;
  if (!within(T, kMaxRows) || !within(k, sk::kMaxChoices) || !within(R, kMaxRows) || !within(D, sk::kMaxN)) return SK_ERR_ARG;
  if (offsets && !within(E, sk::kMaxExperts)) return SK_ERR_ARG;
  const int64_t e = size_of(elem);
  if (misaligned(y, (uintptr_t)e) || misaligned(dout, (uintptr_t)e) || misaligned(dy, 16) || misaligned(slots, 4) ||
      misaligned(weights, 4) || misaligned(offsets, 4) || misaligned(dweights, 4))
    return SK_ERR_ALIGN;
  if (clash({{dweights ? y : nullptr, R * D * e}, {dout, T * D * e}, {slots, 4 * T * k}, {weights, 4 * T * k},
             {offsets, 4 * (E + 1)}},
            {{dy, R * D * e}, {dweights, 4 * T * k}}))
    return SK_ERR_ARG;
  int dev = 0, cus = 0;
  const sk_status st = sk::host::device_for((hipStream_t)stream, &dev, &cus);
  if (st != SK_OK) return st;
  sk::CombineGradArgs a;
  std::memset(&a, 0, sizeof(a));
  a.dout = dout;
  a.y = y;
  a.slots = slots;
  a.weights = weights;
  a.offsets = offsets;
  a.dy = dy;
  a.dweights = dweights;
  a.T = T;
  a.R = (int)R;
  a.D = (int)D;
  a.k = (int)k;
  a.E = offsets ? (int)E : 0;
  return ok(sk::launch_combine_gradient(a, elem, (hipStream_t)stream));
}

sk_status sk_gemm_grouped(const void* A, const void* B, sk_elem elem, const int32_t* offsets, const int32_t* rows,
                          const void* bias, void* C, int64_t R, int64_t T, int64_t E, int64_t N, int64_t K,
                          int tail_zero, void* stream) {
  if (!half_ok(elem) || !A || !B || !offsets || !C) return SK_ERR_ARG;
  if (!within(R, kMaxRows - 1) || !within(T, kMaxRows - 1) || !within(E, sk::kMaxExperts) || !within(N, sk::kMaxN) ||
      !within(K, sk::kMaxK))
    return SK_ERR_ARG;
  if (rows ? T * K * 2 >= kMaxGathered : T != R) return SK_ERR_ARG;
  if (K % 8 || misaligned(A, 16) || misaligned(B, 16) || misaligned(C, 2) || misaligned(bias, 2) ||
      misaligned(offsets, 4) || misaligned(rows, 4))
    return SK_ERR_ALIGN;
  if (clash({{A, 2 * T * K}, {B, 2 * E * N * K}, {offsets, 4 * (E + 1)}, {rows, 4 * R}, {bias, 2 * E * N}}, {{C, 2 * R * N}}))
    return SK_ERR_ARG;
  int dev = 0, cus = 0;
  const sk_status st = sk::host::device_for((hipStream_t)stream, &dev, &cus);
  if (st != SK_OK) return st;
  sk::GroupedGemm g;
  std::memset(&g, 0, sizeof(g));
  g.P = (const uint8_t*)A;
  g.Q = (const uint8_t*)B;
  g.offsets = offsets;
  g.rows = rows;
  g.bias = (const uint16_t*)bias;
  g.C = (uint16_t*)C;
  g.E = (int)E;
  g.R = (int)R;
  g.S = (int)K;
  g.Nout = (int)N;
  g.p_pitch = g.q_pitch = (int)(2 * K);
  g.p_rows = (int)T;
  g.tail = tail_zero != 0;
  hipStream_t s = (hipStream_t)stream;
  return ok(elem == SK_ELEM_BF16 ? sk::launch_grouped_bf16(g, 0, cus, s) : sk::launch_grouped_f16(g, 0, cus, s));
}

sk_status sk_gemm_grouped_backward(const void* dC, const void* A, const void* B, sk_elem elem, const int32_t* offsets,
                                   const int32_t* rows, void* dA, void* dB, void* dbias, int64_t R, int64_t T, int64_t E,
                                   int64_t N, int64_t K, void* stream) {
  if (!half_ok(elem) || !dC || !offsets || (!dA && !dB && !dbias)) return SK_ERR_ARG;
  if ((dA && !B) || ((dB || dbias) && !A)) return SK_ERR_ARG;
  if (!within(R, kMaxRows - 1) || !within(T, kMaxRows - 1) || !within(E, sk::kMaxExperts) || !within(N, sk::kMaxK) ||
      !within(K, sk::kMaxK))
    return SK_ERR_ARG;
  if (rows ? T * K * 2 >= kMaxGathered : T != R) return SK_ERR_ARG;
  if (K % 8 || N % 8 || misaligned(dC, 16) || misaligned(A, 16) || misaligned(B, 16) || misaligned(dA, 2) ||
      misaligned(dB, 2) || misaligned(dbias, 2) || misaligned(offsets, 4) || misaligned(rows, 4))
    return SK_ERR_ALIGN;
  if (clash({{dC, 2 * R * N}, {dB || dbias ? A : nullptr, 2 * T * K}, {dA ? B : nullptr, 2 * E * N * K},
             {offsets, 4 * (E + 1)}, {rows, 4 * R}},
            {{dA, 2 * R * K}, {dB, 2 * E * N * K}, {dbias, 2 * E * N}}))
    return SK_ERR_ARG;
  int dev = 0, cus = 0;
  const sk_status st = sk::host::device_for((hipStream_t)stream, &dev, &cus);
  if (st != SK_OK) return st;
  sk::GroupedGemm g;
  std::memset(&g, 0, sizeof(g));
  g.P = (const uint8_t*)dC;
  g.offsets = offsets;
  g.E = (int)E;
  g.R = (int)R;
  g.p_pitch = (int)(2 * N);
  g.q_pitch = (int)(2 * K);
  g.Nout = (int)K;
  hipStream_t s = (hipStream_t)stream;
  const auto go = elem == SK_ELEM_BF16 ? sk::launch_grouped_bf16 : sk::launch_grouped_f16;
  if (dA) {
    sk::GroupedGemm a = g;
    a.Q = (const uint8_t*)B;
    a.C = (uint16_t*)dA;
    a.S = (int)N;
    a.tail = 1;
    if (go(a, 1, cus, s) != hipSuccess) return SK_ERR_HIP;
  }
  if (dB || dbias) {
    g.Q = (const uint8_t*)A;
    g.rows = rows;
    g.q_rows = (int)T;
    g.C = (uint16_t*)dB;
    g.dbias = (uint16_t*)dbias;
    g.Mout = (int)N;
    return ok(go(g, 2, cus, s));
  }
  return SK_OK;
}

sk_status sk_quantize_w4(const void* w, sk_elem elem, void* q, void* scale, sk_elem scale_elem, uint8_t* zero, int64_t E,
                         int64_t N, int64_t K, int64_t group, void* stream) {
  if (!elem_ok(elem) || !half_ok(scale_elem) || !w || !q || !scale) return SK_ERR_ARG;
  if (group != 32 && group != 64 && group != 128) return SK_ERR_ARG;
  if (!within(E, sk::kMaxExperts) || !within(N, sk::kMaxN) || !within(K, sk::kMaxK) || K % group) return SK_ERR_ARG;
  if (misaligned(w, (uintptr_t)size_of(elem)) || misaligned(q, 16) || misaligned(scale, 2)) return SK_ERR_ALIGN;
  const int64_t n = E * N * K, groups = n / group;
  if (clash({{w, n * size_of(elem)}}, {{q, n / 2}, {scale, 2 * groups}, {zero, groups}})) return SK_ERR_ARG;
  int dev = 0, cus = 0;
  const sk_status st = sk::host::device_for((hipStream_t)stream, &dev, &cus);
  if (st != SK_OK) return st;
  sk::Quant4Args a;
  std::memset(&a, 0, sizeof(a));
  a.w = w;
  a.q = (uint8_t*)q;
  a.scale = scale;
  a.zero = zero;
  a.E = (int)E;
  a.N = (int)N;
  a.K = (int)K;
  a.group = (int)group;
  return ok(sk::launch_quantize_w4(a, elem, scale_elem == SK_ELEM_F16, cus, (hipStream_t)stream));
}

sk_status sk_dequantize_w4(const void* q, const void* scale, sk_elem scale_elem, const uint8_t* zero, void* out,
                           int64_t E, int64_t N, int64_t K, int64_t group, void* stream) {
  if (!half_ok(scale_elem) || !q || !scale || !out) return SK_ERR_ARG;
  if (group != 32 && group != 64 && group != 128) return SK_ERR_ARG;
  if (!within(E, sk::kMaxExperts) || !within(N, sk::kMaxN) || !within(K, sk::kMaxK) || K % group) return SK_ERR_ARG;
  if (misaligned(q, 16) || misaligned(scale, 2) || misaligned(out, 16)) return SK_ERR_ALIGN;
  const int64_t n = E * N * K, groups = n / group;
  if (clash({{q, n / 2}, {scale, 2 * groups}, {zero, groups}}, {{out, 2 * n}})) return SK_ERR_ARG;
  int dev = 0, cus = 0;
  const sk_status st = sk::host::device_for((hipStream_t)stream, &dev, &cus);
  if (st != SK_OK) return st;
  sk::Quant4Args a;
  std::memset(&a, 0, sizeof(a));
  a.q = (uint8_t*)const_cast<void*>(q);
  a.scale = const_cast<void*>(scale);
  a.zero = const_cast<uint8_t*>(zero);
  a.out = out;
  a.E = (int)E;
  a.N = (int)N;
  a.K = (int)K;
  a.group = (int)group;
  return ok(sk::launch_dequantize_w4(a, scale_elem == SK_ELEM_F16, (hipStream_t)stream));
}

sk_status sk_gemm_w4(const void* x, const void* q, const void* scale, const uint8_t* zero, sk_elem elem,
                     const int32_t* offsets, const int32_t* rows, const void* bias, void* C, int64_t M, int64_t T,
                     int64_t E, int64_t N, int64_t K, int64_t group, int tail_zero, void* stream) {
  if (!half_ok(elem) || !x || !q || !scale || !C) return SK_ERR_ARG;
  if (group != 32 && group != 64 && group != 128) return SK_ERR_ARG;
  if (!within(M, kMaxRows - 1) || !within(T, kMaxRows - 1) || !within(E, sk::kMaxExperts) || !within(N, sk::kMaxN) ||
      !within(K, sk::kMaxK) || K % group)
    return SK_ERR_ARG;
  if (offsets ? !rows && T != M : rows || E != 1 || T != M || M > (1 << 20)) return SK_ERR_ARG;
  if (misaligned(x, 16) || misaligned(q, 16) || misaligned(scale, 2) || misaligned(C, 2) || misaligned(bias, 2) ||
      misaligned(offsets, 4) || misaligned(rows, 4))
    return SK_ERR_ALIGN;
  const int64_t n = E * N * K, groups = n / group;
  if (clash({{x, 2 * T * K}, {q, n / 2}, {scale, 2 * groups}, {zero, groups}, {offsets, 4 * (E + 1)}, {rows, 4 * M},
             {bias, 2 * E * N}},
            {{C, 2 * M * N}}))
    return SK_ERR_ARG;
  int dev = 0, cus = 0;
  const sk_status st = sk::host::device_for((hipStream_t)stream, &dev, &cus);
  if (st != SK_OK) return st;
  sk::RowsGemm g;
  std::memset(&g, 0, sizeof(g));
  g.x = (const uint8_t*)x;
  g.W = (const uint8_t*)q;
  g.scale = (const uint8_t*)scale;
  g.zero = zero;
  g.bias = (const uint16_t*)bias;
  g.offsets = offsets;
  g.rows = rows;
  g.C = (uint16_t*)C;
  g.E = (int)E;
  g.R = (int)M;
  g.N = (int)N;
  g.K = (int)K;
  g.x_rows = (int)T;
  g.tail = offsets && tail_zero;
  return ok(sk::launch_rows_w4(g, (int)group, elem == SK_ELEM_F16, cus, (hipStream_t)stream));
}

}  // extern "C"

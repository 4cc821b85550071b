// Routing of tokens to experts and back: the choice of experts with its gradient, the order of rows by expert, and
// the weighted sum of the experts' outputs with its gradients.

#include "sk_experts.h"

namespace sk {

namespace {

// ---------------------------------------------------------------- the choice

// A logit as an integer that orders like it, 0 where it cannot be chosen (-inf, NaN).  (-0 is 0.)
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = f_bits(x + 0.0f);
  const uint32_t k = u ^ ((int32_t)u < 0 ? 0xffffffffu : 0x80000000u);
  return x > -__builtin_inff() ? k : 0u;
}
__device__ __forceinline__ float value_of(uint32_t k) { return bits_f(k ^ ((int32_t)k < 0 ? 0x80000000u : 0xffffffffu)); }

// The largest of L lanes' values, and their sum, in each of the L (a power of two).
template <int L>
__device__ __forceinline__ uint32_t max_of(uint32_t x) {
#pragma unroll
  for (int d = 1; d < L; d *= 2) x = max(x, (uint32_t)__shfl_xor((int)x, d));
  return x;
}
template <int L>
__device__ __forceinline__ float sum_of(float x) {
#pragma unroll
  for (int d = 1; d < L; d *= 2) x += __shfl_xor(x, d);
  return x;
}

// L lanes to a token, V logits to a lane (lane l: l V .. l V + V - 1, so that the first lane that holds the largest key
// holds the lowest expert).  A choice is one maximum over keys; the softmax's maximum is the first choice.
// Counts of a workgroup's pairs by expert go to part [workgroup][E].
template <class T, int L, int V>
__global__ __launch_bounds__(256) void sk_route_choose(RouteArgs a) {
  constexpr int PER = 256 / L;       // tokens at a time
  __shared__ float val[PER][kMaxChoices];
  __shared__ int idx[PER][kMaxChoices];
  __shared__ int count[kMaxExperts];
  const int l = threadIdx.x % L, slot = threadIdx.x / L;
  for (int e = threadIdx.x; e < a.E; e += 256) count[e] = 0;
  __syncthreads();
  const int64_t first = (int64_t)blockIdx.x * a.per_block;
  const int n = (int)min((int64_t)a.per_block, a.T - first);
  for (int at = slot; at < n; at += PER) {
    const int64_t t = first + at;
    const T* const row = (const T*)a.logits + t * a.E;
    uint32_t key[V];
    float x[V];
    bool nan = false;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = l * V + v;
      x[v] = e < a.E ? load_elem(row + e) : -__builtin_inff();
      nan |= x[v] != x[v];
      key[v] = key_of(x[v]);
    }
    float top = 0.0f, total = 0.0f;
    for (int j = 0; j < a.k; ++j) {
      uint32_t best = key[0];
#pragma unroll
      for (int v = 1; v < V; ++v) best = max(best, key[v]);
      const uint32_t most = max_of<L>(best);
      const uint64_t who = __ballot(best == most) >> ((threadIdx.x & 63) / L * L);
      const int winner = __builtin_ctzll(who);            // the first lane of the token's
      int mine = 0;
#pragma unroll
      for (int v = V - 1; v >= 0; --v) mine = key[v] == most ? v : mine;
      if (l == winner) {
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = v == mine ? 0u : key[v];
        idx[slot][j] = most ? l * V + mine : -1;
      }
      const float f = value_of(most);
      if (j == 0) top = f;
      const float p = most ? expf(f - top) : 0.0f;
      if (a.normalize) total += p;
      if (l == 0) val[slot][j] = p;
    }
    if (!a.normalize) {
#pragma unroll
      for (int v = 0; v < V; ++v) total += x[v] > -__builtin_inff() ? expf(x[v] - top) : 0.0f;
      total = sum_of<L>(total);
    }
    nan = (__ballot(nan) >> ((threadIdx.x & 63) / L * L) & (L == 64 ? ~0ull : (1ull << (L & 63)) - 1)) != 0;
    __builtin_amdgcn_wave_barrier();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // (a token's lanes are of one wave)
    for (int j = l; j < a.k; j += L) {
      const int e = idx[slot][j];
      a.experts[t * a.k + j] = e;
      a.weights[t * a.k + j] = e < 0 ? 0.0f : nan ? __builtin_nanf("") : val[slot][j] / total;
      if (e >= 0) atomicAdd(&count[e], 1);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += 256) a.part[(int64_t)blockIdx.x * a.E + e] = count[e];
}

// Lanes of the wave whose key is this lane's, `bits` bits long.
__device__ __forceinline__ uint64_t same_key(int key, int bits) {
  uint64_t m = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const bool on = (key >> b) & 1;
    const uint64_t with = __ballot(on);
    m &= on ? with : ~with;
  }
  return m;
}

// The place of each pair of the workgroup's tokens among all pairs sorted by expert: a stable counting sort.  A
// workgroup adds up the counts of the workgroups before it; a wave takes a run of its pairs, 64 at a time, whose places
// follow from the lanes before it with the same expert.
template <int NT>
__global__ __launch_bounds__(NT) void sk_route_place(RouteArgs a) {
  constexpr int NW = NT / 64;
  extern __shared__ int place_smem[];
  int* const next = place_smem;                 // [NW][E]: a wave's next place in each expert
  int* const scan = place_smem + NW * a.E;      // [NT]
  const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
  const int64_t first = (int64_t)blockIdx.x * a.per_block;
  const int n = (int)(min((int64_t)a.per_block, a.T - first) * a.k);
  const int* const ids = a.experts + first * a.k;
  const int run = ((n + NW - 1) / NW + 63) / 64 * 64;      // pairs of a wave
  const int p0 = min(wave * run, n), p1 = min(p0 + run, n);
  for (int i = threadIdx.x; i < NW * a.E; i += NT) next[i] = 0;
  __syncthreads();
  for (int p = p0 + lane; p < p1; p += 64) {
    const int e = ids[p];
    if (e >= 0) atomicAdd(&next[wave * a.E + e], 1);
  }
  // experts in turn, NT at a time: all workgroups' counts, those before this one, and the sum over experts
  int base = 0;
  for (int e0 = 0; e0 < a.E; e0 += NT) {
    const int e = e0 + (int)threadIdx.x;
    int all = 0, before = 0;
    if (e < a.E) {
      for (int b = 0; b < a.blocks; ++b) {
        const int c = a.part[(int64_t)b * a.E + e];
        all += c;
        before += b < (int)blockIdx.x ? c : 0;
      }
    }
    scan[threadIdx.x] = all;
    __syncthreads();
    for (int d = 1; d < NT; d *= 2) {
      const int y = (int)threadIdx.x >= d ? scan[threadIdx.x - d] : 0;
      __syncthreads();
      scan[threadIdx.x] += y;
      __syncthreads();
    }
    const int upto = base + scan[threadIdx.x];
    if (e < a.E) {
      if (blockIdx.x == 0) {
        if (e == 0) a.offsets[0] = 0;
        a.offsets[e + 1] = upto;
      }
      int at = upto - all + before;
      for (int w = 0; w < NW; ++w) {
        const int c = next[w * a.E + e];
        next[w * a.E + e] = at;
        at += c;
      }
    }
    base += scan[NT - 1];
    __syncthreads();
  }
  const int bits = 32 - __builtin_clz(a.E);       // of keys 0 .. E
  volatile int* const mine = next + wave * a.E;
  for (int p = p0; p < p1; p += 64) {
    const int at = p + lane;
    const int e = at < p1 ? ids[at] : -1;
    const uint64_t same = same_key(e < 0 ? a.E : e, bits);
    const int rank = __popcll(same & ((1ull << lane) - 1));
    int slot = -1;
    if (e >= 0) slot = mine[e] + rank;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_wave_barrier();
    if (e >= 0 && rank == 0) mine[e] = slot + __popcll(same);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_wave_barrier();
    if (at < p1) {
      a.slots[first * a.k + at] = slot;
      if (slot >= 0) a.rows[slot] = (int)(first + at / a.k);
    }
  }
  // rows behind the last expert's belong to no token
  const int64_t all = a.T * a.k;
  for (int64_t r = base + (int64_t)blockIdx.x * NT + threadIdx.x; r < all; r += (int64_t)gridDim.x * NT) a.rows[r] = -1;
}

// dlogits = w (d - sum w d) at the chosen experts, or p (d - sum w d) at all of them (d 0 where not chosen).
template <class T, int L, int V>
__global__ __launch_bounds__(256) void sk_route_gradient(RouteGradArgs a) {
  constexpr int PER = 256 / L;
  const int l = threadIdx.x % L;
  for (int64_t t = (int64_t)blockIdx.x * PER + threadIdx.x / L; t < a.T; t += (int64_t)gridDim.x * PER) {
    const int* const ids = a.experts + t * a.k;
    const float* const w = a.weights + t * a.k;
    const float* const d = a.dweights + t * a.k;
    float x[V], g[V], top = -__builtin_inff(), total = 0.0f, mean = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      g[v] = 0.0f;
      x[v] = 0.0f;
      if (!a.normalize) {
        const int e = l * V + v;
        x[v] = e < a.E ? load_elem((const T*)a.logits + t * a.E + e) : -__builtin_inff();
        top = fmaxf(top, x[v]);
      }
    }
    for (int j = 0; j < a.k; ++j) {
      const int e = ids[j];
      if (e < 0) continue;
      mean = __builtin_fmaf(w[j], d[j], mean);
      if (!a.normalize) {
#pragma unroll
        for (int v = 0; v < V; ++v) g[v] = e == l * V + v ? d[j] : g[v];
      }
    }
    if (a.normalize) {
      for (int j = 0; j < a.k; ++j) {
        const int e = ids[j];
        const float y = w[j] * (d[j] - mean);
#pragma unroll
        for (int v = 0; v < V; ++v) g[v] = e == l * V + v ? y : g[v];
      }
    } else {
#pragma unroll
      for (int d2 = 1; d2 < L; d2 *= 2) top = fmaxf(top, __shfl_xor(top, d2));
#pragma unroll
      for (int v = 0; v < V; ++v) {
        // (a NaN compares false and stays one; a token without a choice has probabilities of 0)
        x[v] = x[v] == -__builtin_inff() ? 0.0f : expf(x[v] - top);
        total += x[v];
      }
      total = sum_of<L>(total);
#pragma unroll
      for (int v = 0; v < V; ++v) g[v] = (total != 0.0f ? x[v] / total : 0.0f) * (g[v] - mean);
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (l * V + v < a.E) store_elem((T*)a.dlogits + t * a.E + l * V + v, g[v]);
  }
}

// ---------------------------------------------------------------- the weighted sum

// out[t] = sum_j w[t][j] y[slots[t][j]], eight columns to a thread, fp32 sums in the order of j.
template <class T, bool SHORT>
__global__ __launch_bounds__(256) void sk_combine(CombineArgs a) {
  const int per_row = (a.D + 7) / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t t = i / per_row;
  if (t >= a.T) return;
  const int col = (int)(i - t * per_row) * 8;
  float x[8] = {};
  for (int j = 0; j < a.k; ++j) {
    const int s = a.slots[t * a.k + j];
    if (s < 0 || s >= a.R) continue;
    const float w = a.weights ? a.weights[t * a.k + j] : 1.0f;
    Vec8<T> y = load8<SHORT>((const T*)a.y + (int64_t)s * a.D, col, a.D);
#pragma unroll
    for (int c = 0; c < 8; ++c) x[c] = __builtin_fmaf(w, y.v[c], x[c]);
  }
  put8((T*)a.out + t * a.D + col, a.D - col, x);
}

// A wave to a pair: dy[slot] = w dout[t] and dweights = <dout[t], y[slot]>.  Rows behind the last expert's are zeros.
template <class T, bool SHORT>
__global__ __launch_bounds__(256) void sk_combine_gradient(CombineGradArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t pairs = a.T * a.k, waves = (int64_t)gridDim.x * 4;
  for (int64_t p = (int64_t)blockIdx.x * 4 + threadIdx.x / 64; p < pairs; p += waves) {
    const int s = a.slots[p];
    if (s < 0 || s >= a.R) {
      if (a.dweights && lane == 0) a.dweights[p] = 0.0f;
      continue;
    }
    const T* const d = (const T*)a.dout + p / a.k * a.D;
    const float w = a.weights ? a.weights[p] : 1.0f;
    float dot = 0.0f;
    for (int col = lane * 8; col < a.D; col += 512) {
      const Vec8<T> x = load8<SHORT>(d, col, a.D);
      if (a.dweights) {
        const Vec8<T> y = load8<SHORT>((const T*)a.y + (int64_t)s * a.D, col, a.D);
#pragma unroll
        for (int c = 0; c < 8; ++c) dot = __builtin_fmaf(x.v[c], y.v[c], dot);
      }
      float v[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) v[c] = w * x.v[c];
      put8((T*)a.dy + (int64_t)s * a.D + col, a.D - col, v);
    }
    if (a.dweights) {
      dot = wave_sum(dot);
      if (lane == 0) a.dweights[p] = dot;
    }
  }
  // (without offsets the launcher has cleared all of dy first)
  if (!a.offsets) return;
  const int64_t from = (int64_t)min(max(a.offsets[a.E], 0), a.R) * a.D, to = (int64_t)a.R * a.D;
  for (int64_t i = from + (int64_t)blockIdx.x * 256 + threadIdx.x; i < to; i += (int64_t)gridDim.x * 256)
    store_elem((T*)a.dy + i, 0.0f);
}

__global__ __launch_bounds__(256) void sk_clear(u32x4* p, int64_t n16, uint8_t* tail, int rest) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n16; i += (int64_t)gridDim.x * 256) p[i] = u32x4{};
  if (blockIdx.x == 0 && (int)threadIdx.x < rest) tail[threadIdx.x] = 0;
}

template <class F>
hipError_t by_elem(int elem, F&& f) {
  if (elem == SK_ELEM_BF16) return f(BfElem{});
  if (elem == SK_ELEM_F16) return f(_Float16{});
  return f(float{});
}

// L lanes and V logits to a lane: four to a lane up to 256 experts.
template <class F>
hipError_t by_experts(int E, F&& f) {
  auto go = [&](auto l, auto v) { return f(l, v); };
  using std::integral_constant;
  if (E <= 16) return go(integral_constant<int, 4>{}, integral_constant<int, 4>{});
  if (E <= 32) return go(integral_constant<int, 8>{}, integral_constant<int, 4>{});
  if (E <= 64) return go(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  if (E <= 128) return go(integral_constant<int, 32>{}, integral_constant<int, 4>{});
  if (E <= 256) return go(integral_constant<int, 64>{}, integral_constant<int, 4>{});
  if (E <= 512) return go(integral_constant<int, 64>{}, integral_constant<int, 8>{});
  return go(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}

int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

// Tokens of a workgroup: 256, and more where there would be over 128 workgroups (each of which reads the counts of all).
int route_per_block(int64_t T) { return (int)(cdiv64(cdiv64(T, 128), 256) * 256); }
int64_t route_blocks(int64_t T) { return cdiv64(T, route_per_block(T)); }

hipError_t launch_route(RouteArgs a, int elem, hipStream_t s) {
  a.per_block = route_per_block(a.T);
  a.blocks = (int)route_blocks(a.T);
  const hipError_t e = by_elem(elem, [&](auto t) {
    return by_experts(a.E, [&](auto l, auto v) {
      return launch(sk_route_choose<decltype(t), decltype(l)::value, decltype(v)::value>, dim3((unsigned)a.blocks), 256, s, a);
    });
  });
  if (e != hipSuccess) return e;
  constexpr int NT = 512;
  void* args[] = {&a};
  const hipError_t r = hipLaunchKernel((const void*)sk_route_place<NT>, dim3((unsigned)a.blocks), dim3(NT), args,
                                       (NT / 64 * a.E + NT) * sizeof(int), s);
  if (r != hipSuccess) (void)hipGetLastError();
  return r;
}

hipError_t launch_route_gradient(const RouteGradArgs& a, int elem, hipStream_t s) {
  return by_elem(elem, [&](auto t) {
    return by_experts(a.E, [&](auto l, auto v) {
      constexpr int L = decltype(l)::value;
      return launch(sk_route_gradient<decltype(t), L, decltype(v)::value>,
                    dim3((unsigned)std::min<int64_t>(cdiv64(a.T, 256 / L), 1 << 20)), 256, s, a);
    });
  });
}

hipError_t launch_combine(const CombineArgs& a, int elem, hipStream_t s) {
  const int64_t blocks = cdiv64(a.T * cdiv64(a.D, 8), 256);
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  return by_elem(elem, [&](auto t) {
    using T = decltype(t);
    return launch(a.D < 8 ? sk_combine<T, true> : sk_combine<T, false>, dim3((unsigned)blocks), 256, s, a);
  });
}

hipError_t launch_combine_gradient(const CombineGradArgs& a, int elem, hipStream_t s) {
  if (!a.offsets) {
    const int64_t bytes = (int64_t)a.R * a.D * (elem == SK_ELEM_F32 ? 4 : 2), n16 = bytes / 16;
    const hipError_t e = launch(sk_clear, dim3((unsigned)std::max<int64_t>(1, std::min<int64_t>(cdiv64(n16, 256), 4096))), 256, s,
                                (u32x4*)a.dy, n16, (uint8_t*)a.dy + n16 * 16, (int)(bytes % 16));
    if (e != hipSuccess) return e;
  }
  const int64_t blocks = std::min<int64_t>(cdiv64(a.T * a.k, 4), 1 << 20);
  return by_elem(elem, [&](auto t) {
    using T = decltype(t);
    return launch(a.D < 8 ? sk_combine_gradient<T, true> : sk_combine_gradient<T, false>, dim3((unsigned)blocks), 256, s, a);
  });
}

}  // namespace sk

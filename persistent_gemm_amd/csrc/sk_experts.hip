// Routing of tokens to experts and back: the choice of experts with its gradient, the order of rows by expert, and
// the weighted sum of the experts' outputs with its gradients.

#include "sk_experts.h"

namespace sk {

namespace {

// ---------------------------------------------------------------- the choice

constexpr int kFewTokens = 64, kPlaceBlocks = 2;

// A logit as an integer that orders like it, 0 where it cannot be chosen (-inf, NaN).  (-0 is 0.)
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = f_bits(x + 0.0f);
  const uint32_t k = u ^ ((int32_t)u < 0 ? 0xffffffffu : 0x80000000u);
  return x > -__builtin_inff() ? k : 0u;
}
__device__ __forceinline__ float value_of(uint32_t k) { return bits_f(k ^ ((int32_t)k < 0 ? 0x80000000u : 0xffffffffu)); }

// f over L lanes' values (a power of two) in each of the L, always in the same order: lanes one and two apart, mirrored halves and
// whole rows of 16, then rows exchanged.
template <int L, class F>
__device__ __forceinline__ uint32_t over_lanes(uint32_t x, F&& f) {
  auto dpp = [](uint32_t v, auto c) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(c)::value, 0xf, 0xf, true); };
  using std::integral_constant;
  if constexpr (L >= 2) x = f(x, dpp(x, integral_constant<int, 0xb1>{}));
  if constexpr (L >= 4) x = f(x, dpp(x, integral_constant<int, 0x4e>{}));
  if constexpr (L >= 8) x = f(x, dpp(x, integral_constant<int, 0x141>{}));
  if constexpr (L >= 16) x = f(x, dpp(x, integral_constant<int, 0x140>{}));
  if constexpr (L >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = f(r[0], r[1]);
  }
  if constexpr (L >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    x = f(r[0], r[1]);
  }
  return x;
}
template <int L>
__device__ __forceinline__ uint32_t max_of(uint32_t x) {
  return over_lanes<L>(x, [](uint32_t a, uint32_t b) { return max(a, b); });
}
// Over the whole wave, in a scalar register: rows' maxima handed on from row to row, up to the last lane's.
template <>
__device__ __forceinline__ uint32_t max_of<64>(uint32_t x) {
  x = max_of<16>(x);
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x142, 0xa, 0xf, false));
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x143, 0xc, 0xf, false));
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}
template <int L>
__device__ __forceinline__ float sum_of(float x) {
  return bits_f(over_lanes<L>(f_bits(x), [](uint32_t a, uint32_t b) { return f_bits(bits_f(a) + bits_f(b)); }));
}
template <int L>
__device__ __forceinline__ float largest_of(float x) {
  return bits_f(over_lanes<L>(f_bits(x), [](uint32_t a, uint32_t b) { return f_bits(fmaxf(bits_f(a), bits_f(b))); }));
}

// V consecutive logits of a row from column `col` on, -inf behind its end.  `wide`: E is a multiple of V and rows are aligned to V
// elements, so that a lane's are all there or none.
template <class T, int V>
__device__ __forceinline__ void load_logits(const T* row, int col, int E, bool wide, float (&x)[V]) {
  if (wide) {
    constexpr int W = V * sizeof(T) / 4 < 4 ? V * sizeof(T) / 4 : 4;      // words of a load
    typedef uint32_t words __attribute__((ext_vector_type(W)));
    constexpr int N = V * sizeof(T) / (4 * W);
    if (col < E) {
      words w[N];
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = ((const words*)(row + col))[i];
      const T* const t = (const T*)w;
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = load_elem(t + v);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = -__builtin_inff();
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = col + v < E ? load_elem(row + col + v) : -__builtin_inff();
  }
}

// ---------------------------------------------------------------- the order by expert

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

template <int NT>
struct PlaceShared {
  int next[NT / 64 * kMaxExperts];   // [wave][expert]: the wave's next place
  int all[kMaxExperts], before[kMaxExperts];
  int sums[NT / 64];
};

// The place of each of a workgroup's n pairs (from pair `first` on, their choices in ids) among all pairs sorted by expert: a stable
// counting sort.  sh.all has all pairs' counts, sh.before those of the workgroups before this one.  A wave takes a run of
// the pairs, 64 at a time, whose places follow from the lanes before it with the same expert.  Returns the number of all pairs.
template <int NT>
__device__ __forceinline__ int place_pairs(const RouteArgs& a, PlaceShared<NT>& sh, const int* ids, int64_t first, int n, bool write_offsets) {
  constexpr int WAVES = NT / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
  const int run = ((n + WAVES - 1) / WAVES + 63) / 64 * 64;      // pairs of a wave
  const int p0 = min(wave * run, n), p1 = min(p0 + run, n);
  for (int i = threadIdx.x; i < WAVES * a.E; i += NT) sh.next[i] = 0;
  __syncthreads();
  for (int p = p0 + lane; p < p1; p += 64) {
    const int e = ids[p];
    if (e >= 0) atomicAdd(&sh.next[wave * a.E + e], 1);
  }
  int base = 0;
  for (int e0 = 0; e0 < a.E; e0 += NT) {
    const int e = e0 + (int)threadIdx.x;
    const int mine = e < a.E ? sh.all[e] : 0;
    int x = mine;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int y = __shfl_up(x, d);
      x += lane >= d ? y : 0;
    }
    if (lane == 63) sh.sums[wave] = x;
    __syncthreads();          // (also: the waves' counts are there)
    int total = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const int s = sh.sums[w];
      x += w < wave ? s : 0;
      total += s;
    }
    if (e < a.E) {
      if (write_offsets) {
        if (e == 0) a.offsets[0] = 0;
        a.offsets[e + 1] = base + x;
      }
      int at = base + x - mine + sh.before[e];
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const int c = sh.next[w * a.E + e];
        sh.next[w * a.E + e] = at;
        at += c;
      }
    }
    base += total;
    __syncthreads();
  }
  const int bits = 32 - __builtin_clz(a.E);       // of keys 0 .. E
  volatile int* const mine = sh.next + wave * a.E;
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
      a.slots[first + at] = slot;
      if (slot >= 0) a.rows[slot] = (int)((uint32_t)(first + at) / (uint32_t)a.k);
    }
  }
  return base;
}

// ---------------------------------------------------------------- the choice

// Choices of the workgroup's tokens, and what is counted of them.  L lanes to a token, V logits to a lane (lane l: l V .. l V + V - 1, so
// that the first lane that holds the largest key holds the lowest expert).  A lane's keys are sorted once (falling, equal ones
// in their order); a choice is then one maximum over the lanes' first keys, and the lane that had it moves its others up.
// The softmax's maximum is the first choice.  Lane l keeps choices l, l + L, ...
template <class T, int L, int V, int NT>
__device__ __forceinline__ void choose(const RouteArgs& a, int64_t first, int n, int* count, int* ids) {
  constexpr int PER = NT / L, KEPT = (kMaxChoices + L - 1) / L;
  const int lane = threadIdx.x & 63, l = threadIdx.x % L, group = lane / L * L;
  const bool wide = a.E % V == 0 && ((uintptr_t)a.logits & (V * sizeof(T) - 1)) == 0;
  for (int at = threadIdx.x / L; at < n; at += PER) {
    const int64_t t = first + at;
    uint32_t key[V];
    int expert[V];
    float x[V];
    load_logits<T, V>((const T*)a.logits + t * a.E, l * V, a.E, wide, x);
    bool nan = false;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      nan |= x[v] != x[v];
      key[v] = key_of(x[v]);
      expert[v] = l * V + v;
    }
#pragma unroll
    for (int round = 0; round < V - 1; ++round)
#pragma unroll
      for (int v = 0; v < V - 1 - round; ++v) {
        const bool swap = key[v + 1] > key[v];
        const uint32_t hi = max(key[v], key[v + 1]), lo = min(key[v], key[v + 1]);
        int above = expert[v + 1], own = expert[v];
        asm volatile("" : "+v"(above), "+v"(own));       // (else the choice of two elements becomes one by an index, several of them for each)
        const int e0 = swap ? above : own, e1 = swap ? own : above;
        key[v] = hi;
        key[v + 1] = lo;
        expert[v] = e0;
        expert[v + 1] = e1;
      }
    uint32_t top_key = 0, kept[KEPT];
    int which[KEPT];
#pragma unroll
    for (int q = 0; q < KEPT; ++q) {
      kept[q] = 0u;
      which[q] = -1;
    }
    // the lane's experts in the order of their keys, four bits each
    std::conditional_t<(V > 8), uint64_t, uint32_t> order = 0;
    static_assert(V <= 16);
#pragma unroll
    for (int v = 0; v < V; ++v) order |= (decltype(order))(expert[v] & 15) << (4 * v);
    for (int j = 0; j < a.k; ++j) {
      // (with a token to a wave all of this is the same in all lanes, and scalar)
      const uint32_t most = max_of<L>(key[0]);
      if (j == 0) top_key = most;
      const int winner = __builtin_ctzll(__ballot(key[0] == most) >> group);            // the first lane of the token's
      const int of = L == 64 ? __builtin_amdgcn_readlane((int)order, winner) : __shfl((int)order, group + winner);
      const int e = winner * V + (of & 15) % V;
      const bool mine = l == winner;
      uint32_t above = 0u;
#pragma unroll
      for (int v = V - 1; v >= 0; --v) {
        const uint32_t own = key[v];
        asm volatile("" : "+v"(above));       // (as in the sort)
        key[v] = mine ? above : own;
        above = own;
      }
      order = mine ? order >> 4 : order;
#pragma unroll
      for (int q = 0; q < KEPT; ++q) {
        const bool here = j == q * L + l;
        kept[q] = here ? most : kept[q];
        which[q] = here ? (most ? e : -1) : which[q];
      }
    }
    const float top = value_of(top_key);
    float p[KEPT], total = 0.0f;
#pragma unroll
    for (int q = 0; q < KEPT; ++q) {
      p[q] = kept[q] ? expf(value_of(kept[q]) - top) : 0.0f;
      total += p[q];
    }
    if (!a.normalize) {
      total = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) total += x[v] > -__builtin_inff() ? expf(x[v] - top) : 0.0f;
    }
    total = sum_of<L>(total);
    nan = (__ballot(nan) >> group & (L == 64 ? ~0ull : (1ull << (L & 63)) - 1)) != 0;
#pragma unroll
    for (int q = 0; q < KEPT; ++q) {
      const int j = q * L + l, e = which[q];
      if (j < a.k) {
        a.experts[t * a.k + j] = e;
        a.weights[t * a.k + j] = e < 0 ? 0.0f : nan ? __builtin_nanf("") : p[q] / total;
        if (ids) ids[at * a.k + j] = e;
        if (e >= 0) atomicAdd(&count[e], 1);
      }
    }
  }
}

// Many tokens: their choices, and counts by expert of each workgroup's, part [workgroup][E].  (16384 x 256
// fp32 logits, 8 chosen: 16.5 us traced by itself; with the places 22.5 us as a call among others.  What bounds it is the issue of
// some 350 vector instructions a token, half of them for the eight maxima; the logits are 16.8 MB, 2.8 us at 6.1 TB/s.)
constexpr int kChooseThreads = 1024, kPlaceThreads = 1024, kFewThreads = 512;
template <class T, int L, int V>
__global__ __launch_bounds__(kChooseThreads) void sk_route_choose(RouteArgs a) {
  __shared__ int count[kMaxExperts];
  for (int e = threadIdx.x; e < a.E; e += kChooseThreads) count[e] = 0;
  __syncthreads();
  const int64_t first = (int64_t)blockIdx.x * a.per_block;
  choose<T, L, V, kChooseThreads>(a, first, (int)min((int64_t)a.per_block, a.T - first), count, nullptr);
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kChooseThreads) a.part[(int64_t)blockIdx.x * a.E + e] = count[e];
}

// The places of the pairs of kPlaceBlocks workgroups of the first kernel; rows behind the last expert's belong to no token.
// (131072 pairs of 256 experts 9.7 us traced: the latency of the counts, of the scan and of the pairs' two readings one after the other.  Every
// workgroup adds up all counts itself, which takes less than a kernel between the two would.)
__global__ __launch_bounds__(kPlaceThreads) void sk_route_place(RouteArgs a) {
  __shared__ PlaceShared<kPlaceThreads> sh;
  for (int e = threadIdx.x; e < a.E; e += kPlaceThreads) sh.all[e] = sh.before[e] = 0;
  __syncthreads();
  // the counts of all workgroups: `wide` threads side by side, the rest shares out the workgroups
  const int wide = a.E >= kPlaceThreads ? kPlaceThreads : 1 << (32 - __builtin_clz(max(a.E - 1, 1)));
  const int lanes = min(wide, kPlaceThreads), share = kPlaceThreads / lanes, b0 = threadIdx.x / lanes;
  const int own = (int)blockIdx.x * kPlaceBlocks;
  for (int e = threadIdx.x % lanes; e < a.E; e += lanes) {
    int all = 0, before = 0;
#pragma unroll 8
    for (int b = b0; b < a.blocks; b += share) {
      const int c = a.part[(int64_t)b * a.E + e];
      all += c;
      before += b < own ? c : 0;
    }
    atomicAdd(&sh.all[e], all);
    atomicAdd(&sh.before[e], before);
  }
  __syncthreads();
  const int64_t first = (int64_t)own * a.per_block;
  const int n = (int)(min((int64_t)a.per_block * kPlaceBlocks, a.T - first) * a.k);
  const int base = place_pairs(a, sh, a.experts + first * a.k, first * a.k, n, blockIdx.x == 0);
  const int64_t all = a.T * a.k;
  for (int64_t r = base + (int64_t)blockIdx.x * kPlaceThreads + threadIdx.x; r < all; r += (int64_t)gridDim.x * kPlaceThreads) a.rows[r] = -1;
}

// Few tokens: both in one workgroup.
template <class T, int L, int V>
__global__ __launch_bounds__(kFewThreads) void sk_route_few(RouteArgs a) {
  __shared__ PlaceShared<kFewThreads> sh;
  __shared__ int ids[kFewTokens * kMaxChoices];
  for (int e = threadIdx.x; e < a.E; e += kFewThreads) sh.all[e] = sh.before[e] = 0;
  __syncthreads();
  choose<T, L, V, kFewThreads>(a, 0, (int)a.T, sh.all, ids);
  __syncthreads();
  const int n = (int)a.T * a.k, base = place_pairs(a, sh, ids, 0, n, true);
  for (int r = base + threadIdx.x; r < n; r += kFewThreads) a.rows[r] = -1;
}

// dlogits = w (d - sum w d) at the chosen experts, or p (d - sum w d) at all of them (d 0 where not chosen).
// (Choice j is read by lane j.  16384 x 256 fp32, 8 chosen, over the chosen 5.2 us and over all 7.6, of which 18 and 35 MB of traffic
// are 3.0 and 5.8; with the choices handed round the wave and compared with each lane's experts a third more.)
template <class T, int L, int V>
__global__ __launch_bounds__(256) void sk_route_gradient(RouteGradArgs a) {
  constexpr int PER = 256 / L, KEPT = (kMaxChoices + L - 1) / L;
  __shared__ __attribute__((aligned(16))) float rows[256 * V];
  const int l = threadIdx.x % L;
  float* const row = rows + threadIdx.x / L * (L * V);       // the token's experts
  const bool wide = a.E % V == 0 && (((uintptr_t)a.logits | (uintptr_t)a.dlogits) & (V * sizeof(T) - 1)) == 0;
  for (int64_t t = (int64_t)blockIdx.x * PER + threadIdx.x / L; t < a.T; t += (int64_t)gridDim.x * PER) {
    float x[V], g[V], w[KEPT], d[KEPT], mean = 0.0f;
    int e[KEPT];
    if (!a.normalize) load_logits<T, V>((const T*)a.logits + t * a.E, l * V, a.E, wide, x);
#pragma unroll
    for (int q = 0; q < KEPT; ++q) {
      const int j = q * L + l;
      const int64_t at = t * a.k + min(j, a.k - 1);      // (three loads that do not wait for one another)
      const int id = a.experts[at];
      w[q] = a.weights[at];
      d[q] = a.dweights[at];
      e[q] = j < a.k ? id : -1;
      if (e[q] >= 0) mean = __builtin_fmaf(w[q], d[q], mean);
    }
    mean = sum_of<L>(mean);
    // (zeros, and then the chosen experts', by way of LDS.  A wave's LDS accesses are done in their order.)
#pragma unroll
    for (int v = 0; v < V; ++v) row[l * V + v] = 0.0f;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int q = 0; q < KEPT; ++q)
      if ((uint32_t)e[q] < (uint32_t)a.E) row[e[q]] = a.normalize ? w[q] * (d[q] - mean) : d[q];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int v = 0; v < V; ++v) g[v] = row[l * V + v];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (!a.normalize) {
      float top = x[0], total = 0.0f;
#pragma unroll
      for (int v = 1; v < V; ++v) top = fmaxf(top, x[v]);
      top = largest_of<L>(top);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        // (a NaN compares false and stays one; a token without a choice has probabilities of 0)
        x[v] = x[v] == -__builtin_inff() ? 0.0f : expf(x[v] - top);
        total += x[v];
      }
      total = sum_of<L>(total);
      const float r = total != 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) g[v] = x[v] * r * (g[v] - mean);
    }
    T* const to = (T*)a.dlogits + t * a.E + l * V;
    if (wide) {
      constexpr int W = V * sizeof(T) / 4 < 4 ? V * sizeof(T) / 4 : 4, N = V * sizeof(T) / (4 * W);
      typedef uint32_t words __attribute__((ext_vector_type(W)));
      words w[N];
#pragma unroll
      for (int v = 0; v < V; ++v) store_elem((T*)w + v, g[v]);
      if (l * V < a.E) {
#pragma unroll
        for (int i = 0; i < N; ++i) ((words*)to)[i] = w[i];
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (l * V + v < a.E) store_elem(to + v, g[v]);
    }
  }
}

// ---------------------------------------------------------------- the weighted sum

// out[t] = sum_j w[t][j] y[slots[t][j]], eight columns to a thread, fp32 sums in the order of j.
// (8192 x 2 x 4096 bf16 39.5 us from memory, 5.1 TB/s, which bounds it; 30 us where y is in the last-level cache.)
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
// (1037 x 4 x 2051 bf16 9.4 us, of which 38 MB of traffic are 6.2.)
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

// Tokens that one workgroup chooses for and places: two turns of its lanes.  (64 of 64 experts 6.0 us and as two kernels 8.0, 32 of 128
// 6.6 / 7.9, 16 of 256 6.3 / 8.0.)
int64_t few_tokens(int E) { return E <= 64 ? kFewTokens : E <= 128 ? kFewTokens / 2 : kFewTokens / 4; }
// Tokens of a workgroup of the first kernel: no more than its waves take at once, and more where there would be over 256 workgroups,
// whose counts are all read by half as many.  (1024 tokens of 256 experts, both kernels, 10.1 us with 16 and 17.9 with 64; of 8
// 8.2 / 8.1.)
int route_per_block(int64_t T, int E) {
  const int least = E <= 32 ? 64 : 16;
  return (int)(cdiv64(cdiv64(T, 256), least) * least);
}
// (none where one workgroup does it all)
int64_t route_blocks(int64_t T, int E) { return T <= few_tokens(E) ? 0 : cdiv64(T, route_per_block(T, E)); }

hipError_t launch_route(RouteArgs a, int elem, hipStream_t s) {
  // one workgroup for few tokens: 1 token of 64 experts 5.2 us against 8.0 as two kernels
  if (a.T <= few_tokens(a.E))
    return by_elem(elem, [&](auto t) {
      return by_experts(a.E, [&](auto l, auto v) {
        return launch(sk_route_few<decltype(t), decltype(l)::value, decltype(v)::value>, dim3(1), kFewThreads, s, a);
      });
    });
  a.per_block = route_per_block(a.T, a.E);
  a.blocks = (int)route_blocks(a.T, a.E);
  const hipError_t e = by_elem(elem, [&](auto t) {
    return by_experts(a.E, [&](auto l, auto v) {
      return launch(sk_route_choose<decltype(t), decltype(l)::value, decltype(v)::value>, dim3((unsigned)a.blocks), kChooseThreads, s, a);
    });
  });
  if (e != hipSuccess) return e;
  return launch(sk_route_place, dim3((unsigned)cdiv64(a.blocks, kPlaceBlocks)), kPlaceThreads, s, a);
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

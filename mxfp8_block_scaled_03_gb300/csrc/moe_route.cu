// moe_route.cu -- the router's decisions in front of a MoE layer, forward and backward: every token's k largest
// logits, their routing weights, the choices per expert, the balance loss and the loss on the logits' scale.
//
// For token t with logits l_te that takes part (its mask is set and some logit is above -inf), N of them in all:
//   lse_t = log sum_e exp(l_te),  p_te = exp(l_te - lse_t)
//   choices: the k largest logits above -inf, the lower expert first among equals
//   gate_tj = p of choice j, divided by the sum over the token's choices with `normalize`
//   count_e = choices of expert e,  P_e = sum_t p_te
//   balance = E sum_e count_e / (N k) * P_e / N,      z = sum_t lse_t^2 / N
// and for the gradients dg of the gates, dP of P, (db, dz) of the two losses, with counts held fixed:
//   c_e = dP_e + db E count_e / (N^2 k)
//   dl_te = p_te (c_e - sum_i p_ti c_i + 2 dz lse_t / N) + the gates' part:
//     normalized: gate_j (dg_j - sum_i gate_i dg_i) at choice j
//     otherwise:  p_te (dg_e [e chosen] - sum_i gate_i dg_i)
// All of it in 32 bits.
//
// What bounds it: latency.  The logits of 32768 tokens and 64 experts are 4 to 8 MB, about a microsecond of the memory's
// time.  A token has L lanes with eight logits each (four up to eight experts), up to 16 tokens share a warp, and many
// experts take two or four warps.  Every lane sorts its logits once, on integer keys that hold the float's order and the
// expert; each of the k rounds is then a maximum over the lanes' first keys.  The column sums stay in registers (a lane
// sees the same experts of every token) and are joined in a fixed order, so that results do not depend on timing: in the
// CTA where one is enough, over a cluster of 16 up to 32 or 64 passes, and by a second kernel, a cluster of eight, beyond.
//
// Measured (replayed; 32768 tokens, 64 experts, 8 choices, bf16): forward 13 us, 10 and 6 for the two kernels alone;
// backward 7.6 us.  16384 tokens, 8 experts, 2 choices, fp32: 6.9 and 3.4 us.  4 tokens, 128 experts: 4.0 us.  As calls
// from Python, on this machine's cores, 20 to 26 and 13 to 16 us: the allocation of the six outputs and the launches.
// With one warp per token, two logits per lane and selection by 32-lane reductions: 28 us forward; 10.2 us backward.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "mx_device.cuh"
#include "mx_internal.h"
#include "mxfp8moe.h"

namespace mx {
namespace {

constexpr int RT_MAX_E = 1024;
constexpr int RT_MAX_K = 32;
constexpr int RT_MAX_CTAS = 304;
constexpr int RT_CLUSTER = 16;         // CTAs of the forward that join their sums without a second kernel
constexpr int RT_FINAL_THREADS = 512;
constexpr uint32_t FULL = 0xFFFFFFFFu;

struct RouteParams {
  const void* logits;
  const uint8_t* mask;
  int64_t T;
  int E, k, normalize, spread;
  int32_t* experts;       // forward: out; backward: in (as the next three)
  float* gates;
  float* lse;
  int32_t* counts;        // [E + 1]: choices per expert, tokens that take part
  float* prob_sum;
  float* losses;
  float2* part;           // [gridDim.x][E + 1] the CTAs' sums of p and counts (integer bits), of lse^2 and of tokens
  int vec;                // the logits' rows can be read V at a time
  int cluster;            // the forward's CTAs are one cluster and join their sums themselves
  const float* dgates;    // backward
  const int32_t* row_of_slot;
  const float* dprob_sum;
  const float* dlosses;
  void* dlogits;
};

__device__ __forceinline__ float load_logit(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const uint16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16);
}
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) {
  *p = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
// V consecutive logits (V a multiple of 4, aligned).
template <int V>
__device__ __forceinline__ void load_logits(const float* p, float* v) {
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    const float4 w = __ldg(reinterpret_cast<const float4*>(p + i));
    v[i] = w.x;
    v[i + 1] = w.y;
    v[i + 2] = w.z;
    v[i + 3] = w.w;
  }
}
template <int V>
__device__ __forceinline__ void load_logits(const uint16_t* p, float* v) {
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p + i));
    v[i] = bf16_lo(w.x);
    v[i + 1] = bf16_hi(w.x);
    v[i + 2] = bf16_lo(w.y);
    v[i + 3] = bf16_hi(w.y);
  }
}
template <int V>
__device__ __forceinline__ void store_logits(float* p, const float* v) {
#pragma unroll
  for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
template <int V>
__device__ __forceinline__ void store_logits(uint16_t* p, const float* v) {
#pragma unroll
  for (int i = 0; i < V; i += 4)
    *reinterpret_cast<uint2*>(p + i) = make_uint2(pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3]));
}

constexpr float LOG2E = 1.4426950408889634f;
// exp(v - top): the difference first, so that logits of the type's lowest value stay finite.
__device__ __forceinline__ float exp_below(float v, float top) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"((v - top) * LOG2E));
  return r;
}

// Candidates: unsigned numbers in the order of the logits (-0 counts as +0) and, among equals, the lowest expert first;
// no two of a token are equal, and 0 is none.  The order of a float is that of its bits with the sign turned over (all of
// them if it is negative); below it stands 65535 - expert: 32 bits for bf16, 48 for float.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t order) {
  return __uint_as_float(order ^ ((order >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
constexpr uint32_t ORDER_MINUS_INF = 0x007FFFFFu;
template <typename S>
struct Key;
template <>
struct Key<float> {
  using type = unsigned long long;
  static __device__ __forceinline__ type make(float v, int e) {
    return (static_cast<type>(order_of(v)) << 32) | (65535u - static_cast<uint32_t>(e));
  }
  static __device__ __forceinline__ float value(type c) { return value_of(static_cast<uint32_t>(c >> 32)); }
  static __device__ __forceinline__ int expert(type c) { return static_cast<int>(65535u - static_cast<uint32_t>(c)); }
  static __device__ __forceinline__ bool real(type c) { return static_cast<uint32_t>(c >> 32) > ORDER_MINUS_INF; }
};
template <>
struct Key<uint16_t> {
  using type = uint32_t;
  static __device__ __forceinline__ type make(float v, int e) {
    return (order_of(v) & 0xFFFF0000u) | (65535u - static_cast<uint32_t>(e));
  }
  static __device__ __forceinline__ float value(type c) {   // (the lower half of a negative value's order is not zero)
    return __uint_as_float(__float_as_uint(value_of(c)) & 0xFFFF0000u);
  }
  static __device__ __forceinline__ int expert(type c) { return static_cast<int>(65535u - (c & 0xFFFFu)); }
  static __device__ __forceinline__ bool real(type c) { return (c >> 16) > (ORDER_MINUS_INF >> 16); }
};

// Sorts c[LO .. LO + N) downwards: Batcher's odd-even merge sort, all of its indexes known to the compiler.
template <typename K>
__device__ __forceinline__ void swap_down(K& a, K& b) {
  const K hi = a > b ? a : b;
  b = a > b ? b : a;
  a = hi;
}
template <int LO, int N, int R, typename K>
__device__ __forceinline__ void merge_down(K* c) {
  if constexpr (2 * R < N) {
    merge_down<LO, N, 2 * R>(c);
    merge_down<LO + R, N, 2 * R>(c);
#pragma unroll
    for (int i = LO + R; i + R < LO + N; i += 2 * R) swap_down(c[i], c[i + R]);
  } else {
    swap_down(c[LO], c[LO + R]);
  }
}
template <int LO, int N, typename K>
__device__ __forceinline__ void sort_down(K* c) {
  if constexpr (N > 1) {
    sort_down<LO, N / 2>(c);
    sort_down<LO + N / 2, N / 2>(c);
    merge_down<LO, N, 1>(c);
  }
}

// The L lanes of a token: part of a warp, or two or four warps, which exchange over shared memory (`s`: 2 x 16 words;
// two buffers in turn, so that one barrier per exchange is enough).  Every lane gets the same result.
template <int L>
struct Group {
  unsigned long long* s;
  int turn;
  __device__ __forceinline__ explicit Group(unsigned long long* scratch) : s(scratch), turn(0) {}
  template <typename V, typename F>
  __device__ __forceinline__ V join(V v, F f) {
#pragma unroll
    for (int o = (L < 32 ? L : 32) / 2; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(FULL, v, o));
    if constexpr (L > 32) {
      unsigned long long* buf = s + 16 * turn;   // a word per warp, whatever its type: groups are not in step
      turn ^= 1;
      const int warp = threadIdx.x >> 5, first = threadIdx.x / L * (L / 32);
      if ((threadIdx.x & 31) == 0) *reinterpret_cast<V*>(buf + warp) = v;
      __syncwarp();                           // (bar.sync counts whole warps, whichever lanes come first)
      asm volatile("bar.sync %0, %1;" ::"r"(1 + static_cast<int>(threadIdx.x) / L), "r"(L) : "memory");
      v = *reinterpret_cast<const V*>(buf + first);
#pragma unroll
      for (int i = 1; i < L / 32; ++i) v = f(v, *reinterpret_cast<const V*>(buf + first + i));
    }
    return v;
  }
  __device__ __forceinline__ float sum(float v) {
    return join(v, [](float a, float b) { return a + b; });
  }
  __device__ __forceinline__ float max(float v) {
    return join(v, [](float a, float b) { return fmaxf(a, b); });
  }
  template <typename K>
  __device__ __forceinline__ K best(K v) {
    return join(v, [](K a, K b) { return a > b ? a : b; });
  }
};

// Sum over the CTA (every thread gets it); s has 32 entries.
template <typename V>
__device__ __forceinline__ V block_sum(V v, V* s) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  __syncthreads();
  if (lane == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < static_cast<int>(blockDim.x >> 5) ? s[lane] : V(0);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}

// The losses from the whole sums; `weighted` is this thread's share of sum_e count_e P_e.
__device__ __forceinline__ void put_losses(const RouteParams& p, float weighted, float z, int n) {
  const float nf = fmaxf(static_cast<float>(n), 1.0f);
  p.counts[p.E] = n;
  p.losses[0] = weighted * (static_cast<float>(p.E) / static_cast<float>(p.k)) / nf / nf;
  p.losses[1] = z / nf;
}

__device__ __forceinline__ uint32_t load_remote(uint32_t cluster_addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// A token has L lanes with V consecutive experts each.  Its choice j is kept by lane j % L; with more than one choice per
// lane (MANY, k > L) a lane has room for all it may get.
template <int L, int V>
struct RouteShape {
  static constexpr int THREADS = 512;
  static constexpr int GROUPS = THREADS / L;
  static constexpr int WARPS = THREADS / 32;
  static constexpr int ROWS = L < 32 ? WARPS : GROUPS;                // sums of p that a CTA keeps per expert
  static constexpr int MOST = L * V < RT_MAX_K ? V : (RT_MAX_K + L - 1) / L;
};
// A lane's logits of token t, -inf where there are none.
template <typename S, int V>
__device__ __forceinline__ void fetch(const RouteParams& p, int64_t t, int e0, bool on, float* v) {
  const S* row = static_cast<const S*>(p.logits) + t * p.E + e0;
  if (p.vec && on && e0 < p.E) {
    load_logits<V>(row, v);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = on && e0 + i < p.E ? load_logit(row + i) : -INFINITY;
  }
}

template <typename S, int L, int V, bool MANY>
__global__ void __launch_bounds__(RouteShape<L, V>::THREADS, 2) k_route_fwd(const RouteParams p) {
  using R = RouteShape<L, V>;
  using K = typename Key<S>::type;
  constexpr int SLOTS = MANY ? R::MOST : 1;
  extern __shared__ float s_dyn[];            // [ROWS][E] sums of p, then [E] counts
  __shared__ unsigned long long s_x[32];
  __shared__ float s_f[32];
  __shared__ int s_i[32];
  Group<L> lanes(s_x);
  const int l = threadIdx.x % L, group = threadIdx.x / L;
  const int E = p.E, k = p.k, e0 = l * V;
  int* hist = reinterpret_cast<int*>(s_dyn + R::ROWS * E);
  for (int e = threadIdx.x; e < E; e += R::THREADS) hist[e] = 0;
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  float psum[V];
#pragma unroll
  for (int i = 0; i < V; ++i) psum[i] = 0.0f;
  float zsum = 0.0f;
  int n = 0;
  float ahead[V];                             // the next token's logits
  auto ask = [&](int64_t t) {
    const bool on = t < p.T && (p.mask == nullptr || p.mask[t] != 0);
    fetch<S, V>(p, t, e0, on, ahead);
  };
  ask(static_cast<int64_t>(blockIdx.x) * R::GROUPS + group);
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * R::GROUPS; t0 < p.T;
       t0 += static_cast<int64_t>(gridDim.x) * R::GROUPS) {
    const int64_t t = t0 + group;
    const bool in = t < p.T;
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = ahead[i];
    ask(t + static_cast<int64_t>(gridDim.x) * R::GROUPS);
    // the largest logit; +inf stands for a NaN or +inf among them: the token's results are NaN
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) top = v[i] < INFINITY ? fmaxf(top, v[i]) : INFINITY;
    top = lanes.max(top);
    const bool odd = top == INFINITY;
    const bool some = top > -INFINITY;
    const float base = some ? top : 0.0f;
    float total = 0.0f;
    K c[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      c[i] = odd || e0 + i >= E ? K(0) : Key<S>::make(v[i], e0 + i);
      v[i] = exp_below(v[i], base);           // 0 for -inf
      total += v[i];
    }
    total = lanes.sum(total);
    if (odd) total = NAN;
    const float inv = some ? 1.0f / total : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) psum[i] = fmaf(v[i], inv, psum[i]);
    const float lse = some ? top + logf(total) : -INFINITY;
    if (in && l == 0) {
      p.lse[t] = odd ? NAN : lse;
      if (some) {
        zsum += odd ? NAN : lse * lse;
        ++n;
      }
    }
    // k rounds: every lane offers the best it has left; the one whose offer is taken moves up
    sort_down<0, V>(c);
    K mine[SLOTS];
    float chosen = 0.0f;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      mine[s] = 0;
#pragma unroll 1
      for (int r = 0; r < L && s * L + r < k; ++r) {
        const K best = lanes.best(c[0]);
        if (l == r) mine[s] = best;
        const bool taken = best == c[0];
#pragma unroll
        for (int i = 0; i + 1 < V; ++i) c[i] = taken ? c[i + 1] : c[i];
        if (taken) c[V - 1] = 0;
      }
      if (Key<S>::real(mine[s])) chosen += exp_below(Key<S>::value(mine[s]), base);
    }
    chosen = lanes.sum(chosen);
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      const int j = s * L + l;
      if (in && j < k) {
        const int64_t slot = t * k + j;
        const bool real = Key<S>::real(mine[s]);
        const int e = Key<S>::expert(mine[s]);
        p.experts[slot] = real ? e : p.spread ? static_cast<int>(static_cast<uint32_t>(slot) % E) : -1;
        p.gates[slot] = real ? exp_below(Key<S>::value(mine[s]), base) / (p.normalize ? chosen : total) : 0.0f;
        if (real) atomicAdd(&hist[e], 1);
      }
    }
  }
  // the CTA's sums: lanes of a warp with the same experts, then the rest in order
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int o = L; o < 32; o <<= 1) psum[i] += __shfl_xor_sync(FULL, psum[i], o);
    if ((L >= 32 || (threadIdx.x & 31) < L) && e0 + i < E)
      s_dyn[(L < 32 ? threadIdx.x >> 5 : group) * E + e0 + i] = psum[i];
  }
  zsum = block_sum(zsum, s_f);
  n = block_sum(n, s_i);
  if (p.cluster) {
    // every CTA adds up a share of the experts over the cluster, the first one the rest
    __shared__ float s_w[RT_CLUSTER];
    __shared__ float s_z;
    __shared__ int s_n;
    for (int e = threadIdx.x; e < E; e += R::THREADS) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < R::ROWS; ++w) s += s_dyn[w * E + e];
      s_dyn[e] = s;
    }
    if (threadIdx.x == 0) {
      s_z = zsum;
      s_n = n;
    }
    cluster_sync_all();
    const uint32_t rank = cluster_cta_rank();
    const int share = (E + RT_CLUSTER - 1) / RT_CLUSTER;
    const int e = static_cast<int>(rank) * share + threadIdx.x;
    float weighted = 0.0f;
    if (static_cast<int>(threadIdx.x) < share && e < E) {
      float s = 0.0f;
      int c = 0;
#pragma unroll
      for (int r = 0; r < RT_CLUSTER; ++r) {
        s += __uint_as_float(load_remote(map_to_cta(s_dyn + e, r)));
        c += static_cast<int>(load_remote(map_to_cta(hist + e, r)));
      }
      p.prob_sum[e] = s;
      p.counts[e] = c;
      weighted = s * static_cast<float>(c);
    }
    weighted = block_sum(weighted, s_f);
    float z = 0.0f;
    int all = 0;
    if (rank == 0 && threadIdx.x < RT_CLUSTER) {
      z = __uint_as_float(load_remote(map_to_cta(&s_z, threadIdx.x)));
      all = static_cast<int>(load_remote(map_to_cta(&s_n, threadIdx.x)));
    }
    if (threadIdx.x == 0) st_remote_u32(map_to_cta(s_w + rank, 0), __float_as_uint(weighted));
    cluster_sync_all();
    if (rank == 0 && threadIdx.x < 32) {
      weighted = threadIdx.x < RT_CLUSTER ? s_w[threadIdx.x] : 0.0f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        z += __shfl_xor_sync(FULL, z, o);
        all += __shfl_xor_sync(FULL, all, o);
        weighted += __shfl_xor_sync(FULL, weighted, o);
      }
      if (threadIdx.x == 0) put_losses(p, weighted, z, all);
    }
    return;
  }
  const bool alone = gridDim.x == 1;
  float2* part = p.part + static_cast<int64_t>(blockIdx.x) * (E + 1);
  float weighted = 0.0f;
  for (int e = threadIdx.x; e < E; e += R::THREADS) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < R::ROWS; ++w) s += s_dyn[w * E + e];
    if (alone) {
      p.prob_sum[e] = s;
      p.counts[e] = hist[e];
      weighted += s * static_cast<float>(hist[e]);
    } else {
      part[e] = make_float2(s, __int_as_float(hist[e]));
    }
  }
  if (alone) {
    weighted = block_sum(weighted, s_f);
    if (threadIdx.x == 0) put_losses(p, weighted, zsum, n);
  } else if (threadIdx.x == 0) {
    part[E] = make_float2(zsum, __int_as_float(n));
  }
}

// Adds the CTAs' sums in a fixed order.  A cluster of eight CTAs, each with an eighth of the experts: thread (e, s) takes
// CTAs s, s + slices, ..., a tree joins the slices, and the first CTA gets the others' shares of the balance loss.  (One CTA
// for all took 10 us for 64 experts and 50 for 1024.)
constexpr int RT_FINAL_CTAS = 8;
__global__ void __launch_bounds__(RT_FINAL_THREADS) k_route_final(const RouteParams p, int ctas) {
  __shared__ float s_p[RT_FINAL_THREADS];
  __shared__ int s_c[RT_FINAL_THREADS];
  __shared__ float s_f[32];
  __shared__ int s_i[32];
  __shared__ float s_w[RT_FINAL_CTAS];
  const uint32_t rank = cluster_cta_rank();
  const int share = (p.E + RT_FINAL_CTAS - 1) / RT_FINAL_CTAS;
  int width = 1;
  while (width < share) width <<= 1;
  const int slices = RT_FINAL_THREADS / width;
  const int own = threadIdx.x % width, slice = threadIdx.x / width;
  const int e = static_cast<int>(rank) * share + own;
  const bool in = own < share && e < p.E;
  // The first CTA's shared memory is written below, by the soonest (one without experts) at once: it has to run by then.
  // While the kernel before this one is still at work the barrier costs nothing.
  cluster_sync_all();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float2 zn = make_float2(0.0f, 0.0f);
  for (int i = threadIdx.x; rank == 0 && i < ctas; i += RT_FINAL_THREADS) {
    const float2 o = __ldcg(p.part + static_cast<int64_t>(i) * (p.E + 1) + p.E);
    zn.x += o.x;
    zn.y = __int_as_float(__float_as_int(zn.y) + __float_as_int(o.y));
  }
  float s = 0.0f;
  int c = 0;
  if (in) {
#pragma unroll 8
    for (int i = slice; i < ctas; i += slices) {
      const float2 o = __ldcg(p.part + static_cast<int64_t>(i) * (p.E + 1) + e);
      s += o.x;
      c += __float_as_int(o.y);
    }
  }
  s_p[threadIdx.x] = s;
  s_c[threadIdx.x] = c;
  __syncthreads();
  for (int o = slices / 2; o > 0; o >>= 1) {
    if (slice < o) {
      s_p[threadIdx.x] += s_p[threadIdx.x + o * width];
      s_c[threadIdx.x] += s_c[threadIdx.x + o * width];
    }
    __syncthreads();
  }
  float weighted = 0.0f;
  if (slice == 0 && in) {
    p.prob_sum[e] = s_p[own];
    p.counts[e] = s_c[own];
    weighted = s_p[own] * static_cast<float>(s_c[own]);
  }
  weighted = block_sum(weighted, s_f);
  if (threadIdx.x == 0) st_remote_u32(map_to_cta(s_w + rank, 0), __float_as_uint(weighted));
  cluster_sync_all();
  if (rank == 0) {
    const float z = block_sum(zn.x, s_f);
    const int n = block_sum(__float_as_int(zn.y), s_i);
    if (threadIdx.x == 0) {
      float all = 0.0f;
      for (int i = 0; i < RT_FINAL_CTAS; ++i) all += s_w[i];
      put_losses(p, all, z, n);
    }
  }
}

// What a token's lane reads in the backward: asked for one token ahead.
template <int V, int SLOTS>
struct BwdToken {
  float v[V];
  float lse;
  float g[SLOTS], dg[SLOTS];
  int at[SLOTS];
};

template <typename S, int L, int V, bool MANY>
__global__ void __launch_bounds__(RouteShape<L, V>::THREADS, 2) k_route_bwd(const RouteParams p) {
  using R = RouteShape<L, V>;
  constexpr int SLOTS = MANY ? R::MOST : 1;
  __shared__ unsigned long long s_x[32];
  __shared__ __align__(16) float s_add[MANY ? 1 : R::GROUPS][L * V];
  Group<L> lanes(s_x);
  const int l = threadIdx.x % L, group = threadIdx.x / L;
  const int E = p.E, k = p.k, e0 = l * V;
  if (!MANY) {
    for (int i = threadIdx.x; i < R::GROUPS * L * V; i += R::THREADS) s_add[0][i] = 0.0f;
    __syncthreads();
  }
  const int64_t slots = p.T * k;
  auto ask = [&](int64_t t) {
    BwdToken<V, SLOTS> a;
    const bool in = t < p.T;
    a.lse = in ? __ldg(p.lse + t) : -INFINITY;
    fetch<S, V>(p, t, e0, in, a.v);
#pragma unroll
    for (int q = 0; q < SLOTS; ++q) {
      const int j = q * L + l;
      a.g[q] = a.dg[q] = 0.0f;
      a.at[q] = -1;
      if (in && j < k && p.dgates != nullptr) {
        const int64_t slot = t * k + j;
        a.at[q] = __ldg(p.experts + slot);
        a.g[q] = __ldg(p.gates + slot);
        int64_t from = slot;
        if (p.row_of_slot != nullptr) from = __ldg(p.row_of_slot + slot);
        if (from >= 0 && from < slots) a.dg[q] = __ldg(p.dgates + from);
      }
    }
    return a;
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * R::GROUPS;
  int64_t t = static_cast<int64_t>(blockIdx.x) * R::GROUPS + group;
  BwdToken<V, SLOTS> next;
  if (!MANY) next = ask(t);                   // (with many choices per lane there are no registers for it)
  const float n = fmaxf(static_cast<float>(__ldg(p.counts + E)), 1.0f);
  const float db = p.dlosses != nullptr ? __ldg(p.dlosses) : 0.0f;
  const float dz = p.dlosses != nullptr ? __ldg(p.dlosses + 1) : 0.0f;
  const float unit = db * (static_cast<float>(E) / static_cast<float>(k)) / n / n;
  float c[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    c[i] = e0 + i < E ? unit * static_cast<float>(__ldg(p.counts + e0 + i)) : 0.0f;
    if (e0 + i < E && p.dprob_sum != nullptr) c[i] += __ldg(p.dprob_sum + e0 + i);
  }
  S* dlogits = static_cast<S*>(p.dlogits);
  for (; t - group < p.T; t += step) {
    BwdToken<V, SLOTS> a = MANY ? ask(t) : next;
    if (!MANY) next = ask(t + step);
    const bool on = !(a.lse == -INFINITY);    // the forward leaves -inf where a token takes no part
    // a lane's choices: gate_j dg_j, and where it goes; a gate of 0 passes nothing on, whatever its gradient's place holds
    float gd[SLOTS];
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < SLOTS; ++q) {
      const bool real = on && a.at[q] >= 0 && a.at[q] < E && a.g[q] != 0.0f;
      if (!real) a.at[q] = -1;
      gd[q] = real ? a.g[q] * a.dg[q] : 0.0f;
      s += gd[q];
    }
    s = lanes.sum(s);
    const float lse0 = on ? a.lse : 0.0f;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      a.v[i] = on && e0 + i < E ? exp_below(a.v[i], lse0) : 0.0f;   // p
      dot = fmaf(a.v[i], c[i], dot);
    }
    dot = lanes.sum(dot);
    const float base = on ? 2.0f * dz / n * a.lse - dot - (p.normalize ? 0.0f : s) : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) a.v[i] *= c[i] + base;
    if (p.dgates != nullptr) {
      if constexpr (!MANY) {
        // The choices' shares go through the token's row of shared memory, which is zero but for them: one store, the
        // lane's own V values, one store of zero.  Experts that a token lists more than once are joined first.
        float add = p.normalize ? gd[0] - a.g[0] * s : gd[0];
        const int mine = a.at[0];
        bool put = mine >= 0;
        if (threadIdx.x % L < 32) {           // the choices' lanes are in the group's first warp
          const uint32_t same = __match_any_sync(FULL, put ? group * RT_MAX_E + mine : -1 - static_cast<int>(threadIdx.x));
          if (__any_sync(FULL, (same & (same - 1)) != 0)) {
            float all = 0.0f;
            for (int r = 0; r < 32; ++r) {    // in the order of the slots
              const float o = __shfl_sync(FULL, add, r);
              if ((same >> r) & 1u) all += o;
            }
            add = all;
            put = put && (same & ((1u << (threadIdx.x & 31)) - 1u)) == 0;
          }
        }
        float* row = s_add[group];
        __syncwarp();
        if (put) row[mine] = add;
        if constexpr (L > 32) lanes.sum(0.0f);   // (a barrier of the group)
        else __syncwarp();
#pragma unroll
        for (int i = 0; i < V; i += 4) {
          const float4 o = *reinterpret_cast<const float4*>(row + e0 + i);
          a.v[i] += o.x;
          a.v[i + 1] += o.y;
          a.v[i + 2] += o.z;
          a.v[i + 3] += o.w;
        }
        if constexpr (L > 32) lanes.sum(0.0f);
        else __syncwarp();
        if (put) row[mine] = 0.0f;
      } else {
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) {
          const float add = p.normalize ? gd[q] - a.g[q] * s : gd[q];
          for (int r = 0; r < L && q * L + r < k; ++r) {
            const float o = __shfl_sync(FULL, add, r, L);
            const int e = __shfl_sync(FULL, a.at[q], r, L) - e0;
#pragma unroll
            for (int i = 0; i < V; ++i)
              if (e == i) a.v[i] += o;
          }
        }
      }
    }
    if (t < p.T) {
      S* row = dlogits + t * E + e0;
      if (p.vec) {
        if (e0 < E) store_logits<V>(row, a.v);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (e0 + i < E) store_logit(row + i, a.v[i]);
      }
    }
  }
}

// ---- host side -------------------------------------------------------------------------------

int route_sms() {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> sms[kMaxDevices] = {};
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  if ((n = sms[dev].load()) <= 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 0;
    sms[dev].store(n);
  }
  return n;
}

// Calls f with the lanes and logits per lane of a token: eight logits per lane, so that up to 16 tokens share a warp's
// rounds and a token of many experts has two or four warps.
template <typename F>
auto with_shape(int E, F f) {
  using std::integral_constant;
  if (E <= 4) return f(integral_constant<int, 1>{}, integral_constant<int, 4>{});
  if (E <= 8) return f(integral_constant<int, 2>{}, integral_constant<int, 4>{});
  if (E <= 16) return f(integral_constant<int, 2>{}, integral_constant<int, 8>{});
  if (E <= 32) return f(integral_constant<int, 4>{}, integral_constant<int, 8>{});
  if (E <= 64) return f(integral_constant<int, 8>{}, integral_constant<int, 8>{});
  if (E <= 128) return f(integral_constant<int, 16>{}, integral_constant<int, 8>{});
  if (E <= 256) return f(integral_constant<int, 32>{}, integral_constant<int, 8>{});
  if (E <= 512) return f(integral_constant<int, 64>{}, integral_constant<int, 8>{});
  return f(integral_constant<int, 128>{}, integral_constant<int, 8>{});
}
int groups_of(int E) {
  return with_shape(E, [](auto l, auto v) { return RouteShape<decltype(l)::value, decltype(v)::value>::GROUPS; });
}

// One CTA up to two passes (a token per group each); then a cluster of 16, which leaves most of the GPU idle but needs no
// second kernel; then as many CTAs as give all of them equal passes, and a second kernel for their sums.  The second launch
// costs the call from Python 2.4 to 4.5 us; the cluster's passes cost the GPU more and more.  Replayed, us, the cluster and
// the second kernel, by passes:
//                  16            32            48            64
//   E 8, k 2     4.1  5.7      5.3  5.9      5.8  5.6      6.6  5.7
//   E 8, k 8     5.3  6.6      7.0  6.7      9.2  6.9     10.9  6.7
//   E 64, k 2    5.0  6.0      6.2  6.1      7.4  6.2      8.5  6.0
//   E 64, k 8    5.3  6.4      7.2  6.6      8.7  6.5     10.5  6.6
//   E 256, k 8   5.8  6.8      8.0  7.2      9.8  7.4     11.8  7.6
// So 32 passes, where the cluster costs a replay at most a third of what it saves the call, and 64 for tokens whose passes
// are short: up to eight experts and two rounds.
int cluster_passes(int E, int k) { return (E <= 8 && k <= 2 ? 4 : 2) * RT_CLUSTER; }
struct FwdGrid {
  int ctas;
  bool cluster;
};
FwdGrid fwd_grid(int64_t T, int E, int k, bool clusters) {
  const int64_t passes = (T + groups_of(E) - 1) / groups_of(E);
  if (passes <= 2) return {1, false};
  if (clusters && passes <= cluster_passes(E, k)) return {RT_CLUSTER, true};
  const int64_t most = RT_MAX_CTAS;
  const int64_t per = (passes + most - 1) / most;
  return {static_cast<int>((passes + per - 1) / per), false};
}

bool sizes_ok(int64_t T, int E, int k, int dtype) {
  return T >= 0 && E >= 1 && E <= RT_MAX_E && k >= 1 && k <= E && T <= INT32_MAX / k &&
         (dtype == MOE_LOGITS_BF16 || dtype == MOE_LOGITS_F32);
}
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool logits_ok(const void* p, int dtype) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (dtype == MOE_LOGITS_F32 ? 3u : 1u)) == 0;
}

// Whether clusters of 16 of this kernel can run (asked once per device); a cluster launch.
template <typename F>
cudaLaunchConfig_t cluster_config(F, size_t smem, int threads, cudaLaunchAttribute* attr, cudaStream_t st) {
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = RT_CLUSTER;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(RT_CLUSTER, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}
template <auto KERNEL>
bool clusters_run(size_t smem, int threads) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices] = {};   // 1: no, 2: yes
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
  if (known[dev].load() == 0) {
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = cluster_config(KERNEL, smem, threads, attr, nullptr);
    int n = 0;
    const bool ok =
        cudaFuncSetAttribute(KERNEL, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&n, KERNEL, &cfg) == cudaSuccess && n > 0;
    if (!ok) cudaGetLastError();   // clear: a second kernel joins the sums
    known[dev].store(ok ? 2 : 1);
  }
  return known[dev].load() == 2;
}

// Launches and returns the forward's CTAs that a second kernel has to join (1: none).
template <bool BWD, typename S>
int launch_route(const RouteParams& p, unsigned grid, cudaStream_t st) {
  return with_shape(p.E, [&](auto lanes, auto each) {
    constexpr int L = decltype(lanes)::value, V = decltype(each)::value;
    using R = RouteShape<L, V>;
    RouteParams q = p;
    auto whole = [](const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & (sizeof(S) * 4 - 1)) == 0; };
    q.vec = p.E % V == 0 && whole(p.logits) && (!BWD || whole(p.dlogits));
    auto go = [&](auto many) {
      constexpr bool MANY = decltype(many)::value;
      if constexpr (BWD) {
        k_route_bwd<S, L, V, MANY><<<grid, R::THREADS, 0, st>>>(q);
        return 1;
      } else {
        constexpr auto kernel = k_route_fwd<S, L, V, MANY>;
        const size_t smem = (R::ROWS + 1) * static_cast<size_t>(p.E) * 4;
        FwdGrid g = fwd_grid(p.T, p.E, p.k, true);
        if (g.cluster && !clusters_run<kernel>((R::ROWS + 1) * static_cast<size_t>(L * V) * 4, R::THREADS))
          g = fwd_grid(p.T, p.E, p.k, false);
        if (g.cluster) {
          q.cluster = 1;
          cudaLaunchAttribute attr[1];
          const cudaLaunchConfig_t cfg = cluster_config(kernel, smem, R::THREADS, attr, st);
          cudaLaunchKernelEx(&cfg, kernel, q);
          return 1;
        }
        kernel<<<g.ctas, R::THREADS, smem, st>>>(q);
        return g.ctas;
      }
    };
    if constexpr (R::MOST > 1) {
      if (p.k > L) return go(std::true_type{});
    }
    return go(std::false_type{});
  });
}

}  // namespace
}  // namespace mx

using namespace mx;

extern "C" {

size_t moe_route_workspace_size(int64_t T, int E, int k) {
  if (!sizes_ok(T, E, k, MOE_LOGITS_F32) || k > RT_MAX_K) return 0;
  return static_cast<size_t>(fwd_grid(T, E, k, false).ctas) * (E + 1) * sizeof(float2);
}

int moe_route_fwd(const void* logits, int logits_dtype, int64_t T, int E, int k, const uint8_t* token_mask,
                  int normalize, int spread, int32_t* experts, float* gates, float* lse, int32_t* counts,
                  float* prob_sum, float* losses, void* workspace, size_t workspace_bytes, void* stream) {
  if (!sizes_ok(T, E, k, logits_dtype) || normalize < 0 || normalize > 1 || spread < 0 || spread > 1)
    return MXFP8_ERR_INVALID_ARG;
  if (k > RT_MAX_K) return MXFP8_ERR_UNSUPPORTED;
  if (T > 0 && !logits_ok(logits, logits_dtype)) return MXFP8_ERR_INVALID_ARG;
  for (const void* q : {static_cast<const void*>(experts), static_cast<const void*>(gates),
                        static_cast<const void*>(lse)})
    if ((T > 0 && q == nullptr) || !aligned4(q)) return MXFP8_ERR_INVALID_ARG;
  for (const void* q : {static_cast<const void*>(counts), static_cast<const void*>(prob_sum),
                        static_cast<const void*>(losses)})
    if (q == nullptr || !aligned4(q)) return MXFP8_ERR_INVALID_ARG;
  if (fwd_grid(T, E, k, false).ctas > 1) {
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0) return MXFP8_ERR_INVALID_ARG;
    if (workspace_bytes < moe_route_workspace_size(T, E, k)) return MXFP8_ERR_WORKSPACE;
  }
  RouteParams p{};
  p.logits = logits;
  p.mask = token_mask;
  p.T = T;
  p.E = E;
  p.k = k;
  p.normalize = normalize;
  p.spread = spread;
  p.experts = experts;
  p.gates = gates;
  p.lse = lse;
  p.counts = counts;
  p.prob_sum = prob_sum;
  p.losses = losses;
  p.part = static_cast<float2*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int ctas = logits_dtype == MOE_LOGITS_F32 ? launch_route<false, float>(p, 0, st)
                                                  : launch_route<false, uint16_t>(p, 0, st);
  if (cudaGetLastError() != cudaSuccess) return MXFP8_ERR_CUDA;
  if (ctas > 1) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = RT_FINAL_CTAS;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(RT_FINAL_CTAS, 1, 1);
    cfg.blockDim = dim3(RT_FINAL_THREADS, 1, 1);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, k_route_final, p, ctas) != cudaSuccess) return MXFP8_ERR_CUDA;
  }
  return MXFP8_OK;
}

int moe_route_bwd(const void* logits, int logits_dtype, int64_t T, int E, int k, const int32_t* experts,
                  const float* gates, const float* lse, const int32_t* counts, const float* dgates,
                  const int32_t* row_of_slot, const float* dprob_sum, const float* dlosses, int normalize,
                  void* dlogits, void* stream) {
  if (!sizes_ok(T, E, k, logits_dtype) || normalize < 0 || normalize > 1) return MXFP8_ERR_INVALID_ARG;
  if (row_of_slot != nullptr && dgates == nullptr) return MXFP8_ERR_INVALID_ARG;
  if (k > RT_MAX_K) return MXFP8_ERR_UNSUPPORTED;
  if (T == 0) return MXFP8_OK;
  if (!logits_ok(logits, logits_dtype) || !logits_ok(dlogits, logits_dtype)) return MXFP8_ERR_INVALID_ARG;
  for (const void* q : {static_cast<const void*>(experts), static_cast<const void*>(gates),
                        static_cast<const void*>(lse), static_cast<const void*>(counts)})
    if (q == nullptr || !aligned4(q)) return MXFP8_ERR_INVALID_ARG;
  for (const void* q : {static_cast<const void*>(dgates), static_cast<const void*>(row_of_slot),
                        static_cast<const void*>(dprob_sum), static_cast<const void*>(dlosses)})
    if (!aligned4(q)) return MXFP8_ERR_INVALID_ARG;
  const int sms = route_sms();
  if (sms <= 0) return MXFP8_ERR_CUDA;
  RouteParams p{};
  p.logits = logits;
  p.T = T;
  p.E = E;
  p.k = k;
  p.normalize = normalize;
  p.experts = const_cast<int32_t*>(experts);
  p.gates = const_cast<float*>(gates);
  p.lse = const_cast<float*>(lse);
  p.counts = const_cast<int32_t*>(counts);
  p.dgates = dgates;
  p.row_of_slot = row_of_slot;
  p.dprob_sum = dprob_sum;
  p.dlosses = dlosses;
  p.dlogits = dlogits;
  const int64_t groups = groups_of(E);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>((T + groups - 1) / groups, 2 * sms));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (logits_dtype == MOE_LOGITS_F32) launch_route<true, float>(p, grid, st);
  else launch_route<true, uint16_t>(p, grid, st);
  return cudaGetLastError() == cudaSuccess ? MXFP8_OK : MXFP8_ERR_CUDA;
}

}  // extern "C"

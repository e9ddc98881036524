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
// What bounds it: latency.  The logits of 32768 tokens and 64 experts are 4 to 8 MB, about a microsecond of
// the memory's time.  A group of L lanes (a power of two, at least E up to 32) holds a token, E / L logits
// per lane: the selection is k rounds of an argmax over the group, on integer keys in the order of the floats.
// The column sums stay in registers (a lane sees the same experts of every token); each CTA writes its
// own and a second kernel adds them in a fixed order, so that results do not depend on timing.  A call of few
// tokens is one CTA, which finishes by itself.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>

#include "mx_device.cuh"
#include "mx_internal.h"
#include "mxfp8moe.h"

namespace mx {
namespace {

constexpr int RT_THREADS = 256;
constexpr int RT_WARPS = RT_THREADS / 32;
constexpr int RT_MAX_E = 1024;
constexpr int RT_MAX_K = 32;
constexpr int RT_MAX_CTAS = 304;
constexpr int RT_FINAL_THREADS = 1024;
constexpr uint32_t FULL = 0xFFFFFFFFu;
constexpr uint32_t KEY_MINUS_INF = 0x007FFFFFu;   // route_key(-inf); a key of 0 is no logit at all

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
  float* part_p;          // [gridDim.x][E] the CTAs' sums of p
  int32_t* part_c;        // [gridDim.x][E] and counts
  float* part_z;          // [gridDim.x]
  int32_t* part_n;        // [gridDim.x]
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

// Unsigned keys in the order of the floats (-0 counts as +0).
__device__ __forceinline__ uint32_t route_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float route_value(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// Sums and maxima over a group of L lanes, in an order that every lane shares.
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}
template <int L>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
  return v;
}
template <int L>
__device__ __forceinline__ bool group_any(bool v) {
  const uint32_t b = __ballot_sync(FULL, v);
  return ((b >> ((threadIdx.x & 31) / L * L)) & (L == 32 ? FULL : (1u << (L % 32)) - 1u)) != 0;
}
// Largest key of the group and, among equals, the lowest expert.
template <int L>
__device__ __forceinline__ void group_best(uint32_t& key, int& e) {
  if constexpr (L == 32) {
    const uint32_t top = __reduce_max_sync(FULL, key);
    e = static_cast<int>(__reduce_min_sync(FULL, key == top ? static_cast<uint32_t>(e) : FULL));
    key = top;
  } else {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) {
      const uint32_t other = __shfl_xor_sync(FULL, key, o);
      const int oe = __shfl_xor_sync(FULL, e, o);
      if (other > key || (other == key && oe < e)) {
        key = other;
        e = oe;
      }
    }
  }
}

// Sum over the CTA (every thread gets it); s has RT_FINAL_THREADS / 32 entries.
template <typename V>
__device__ __forceinline__ V block_sum(V v, V* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  V t = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) t += s[w];
  return t;
}

// The losses from the whole sums; `weighted` is this thread's share of sum_e count_e P_e.
__device__ __forceinline__ void put_losses(const RouteParams& p, float weighted, float z, int n) {
  const float nf = fmaxf(static_cast<float>(n), 1.0f);
  p.counts[p.E] = n;
  p.losses[0] = weighted * (static_cast<float>(p.E) / static_cast<float>(p.k)) / nf / nf;
  p.losses[1] = z / nf;
}

// A lane's logits are those of experts l, l + L, ..., l + (V - 1) L.
template <typename S, int L, int V>
__global__ void __launch_bounds__(RT_THREADS) k_route_fwd(const RouteParams p) {
  extern __shared__ float s_dyn[];            // [RT_WARPS][E] sums of p, then [E] counts
  __shared__ float s_f[RT_FINAL_THREADS / 32];
  __shared__ int s_i[RT_FINAL_THREADS / 32];
  constexpr int G = RT_THREADS / L;
  const int l = threadIdx.x % L, group = threadIdx.x / L;
  const int E = p.E, k = p.k;
  int* hist = reinterpret_cast<int*>(s_dyn + RT_WARPS * E);
  for (int e = threadIdx.x; e < E; e += RT_THREADS) hist[e] = 0;
  __syncthreads();
  float psum[V];
#pragma unroll
  for (int i = 0; i < V; ++i) psum[i] = 0.0f;
  float zsum = 0.0f;
  int n = 0;
  const S* logits = static_cast<const S*>(p.logits);
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * G; t0 < p.T; t0 += static_cast<int64_t>(gridDim.x) * G) {
    const int64_t t = t0 + group;
    const bool in = t < p.T;
    const bool on = in && (p.mask == nullptr || p.mask[t] != 0);
    float v[V];
    float top = -INFINITY;
    bool odd = false;                         // a NaN or +inf: the token's results are NaN
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[i] = on && l + L * i < E ? load_logit(logits + t * E + l + L * i) : -INFINITY;
      odd |= !(v[i] < INFINITY);
      top = fmaxf(top, v[i]);
    }
    odd = group_any<L>(odd);
    top = group_max<L>(top);
    const bool some = odd || top > -INFINITY;
    float total = 0.0f;
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      key[i] = some && !odd && l + L * i < E ? route_key(v[i]) : 0u;
      v[i] = some ? expf(v[i] - top) : 0.0f;
      total += v[i];
    }
    total = group_sum<L>(total);
    if (odd) total = NAN;
    const float inv = some ? 1.0f / total : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) psum[i] += v[i] * inv;
    const float lse = some ? top + logf(total) : -INFINITY;
    if (in && l == 0) {
      p.lse[t] = lse;
      if (some) {
        zsum += lse * lse;
        ++n;
      }
    }
    uint32_t mine = 0;                        // lane j keeps choice j
    int mine_e = 0;
    for (int j = 0; j < k; ++j) {
      uint32_t best = 0;
      int e = 0;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == 0 || key[i] > best) {
          best = key[i];
          e = l + L * i;
        }
      group_best<L>(best, e);
      if (l == j) {
        mine = best;
        mine_e = e;
      }
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e == l + L * i) key[i] = 0u;
    }
    const bool real = mine > KEY_MINUS_INF;
    float g = real ? expf(route_value(mine) - top) : 0.0f;
    const float chosen = group_sum<L>(g);
    g = real ? g / (p.normalize ? chosen : total) : 0.0f;
    if (in && l < k) {
      const int64_t slot = t * k + l;
      p.experts[slot] = real ? mine_e : p.spread ? static_cast<int>(static_cast<uint32_t>(slot) % E) : -1;
      p.gates[slot] = g;
      if (real) atomicAdd(&hist[mine_e], 1);
    }
  }
  // the CTA's sums: lanes of a warp with the same experts, then the warps in order
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int o = L; o < 32; o <<= 1) psum[i] += __shfl_xor_sync(FULL, psum[i], o);
    if ((threadIdx.x & 31) < L && l + L * i < E) s_dyn[(threadIdx.x >> 5) * E + l + L * i] = psum[i];
  }
  zsum = block_sum(zsum, s_f);
  n = block_sum(n, s_i);
  const bool alone = gridDim.x == 1;
  float weighted = 0.0f;
  for (int e = threadIdx.x; e < E; e += RT_THREADS) {
    float s = 0.0f;
    for (int w = 0; w < RT_WARPS; ++w) s += s_dyn[w * E + e];
    if (alone) {
      p.prob_sum[e] = s;
      p.counts[e] = hist[e];
      weighted += s * static_cast<float>(hist[e]);
    } else {
      p.part_p[static_cast<int64_t>(blockIdx.x) * E + e] = s;
      p.part_c[static_cast<int64_t>(blockIdx.x) * E + e] = hist[e];
    }
  }
  if (alone) {
    weighted = block_sum(weighted, s_f);
    if (threadIdx.x == 0) put_losses(p, weighted, zsum, n);
  } else if (threadIdx.x == 0) {
    p.part_z[blockIdx.x] = zsum;
    p.part_n[blockIdx.x] = n;
  }
}

// Adds the CTAs' sums in a fixed order: thread (e, s) takes CTAs s, s + slices, ...; then a tree over the slices.
__global__ void __launch_bounds__(RT_FINAL_THREADS) k_route_final(const RouteParams p, int ctas) {
  __shared__ float s_p[RT_FINAL_THREADS];
  __shared__ int s_c[RT_FINAL_THREADS];
  __shared__ float s_f[RT_FINAL_THREADS / 32];
  __shared__ int s_i[RT_FINAL_THREADS / 32];
  int width = 1;
  while (width < p.E) width <<= 1;
  const int slices = RT_FINAL_THREADS / width;
  const int e = threadIdx.x % width, slice = threadIdx.x / width;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float s = 0.0f;
  int c = 0;
  if (e < p.E) {
#pragma unroll 4
    for (int i = slice; i < ctas; i += slices) {
      s += __ldcg(p.part_p + static_cast<int64_t>(i) * p.E + e);
      c += __ldcg(p.part_c + static_cast<int64_t>(i) * p.E + e);
    }
  }
  s_p[threadIdx.x] = s;
  s_c[threadIdx.x] = c;
  const float z = block_sum(threadIdx.x < ctas ? __ldcg(p.part_z + threadIdx.x) : 0.0f, s_f);
  const int n = block_sum(threadIdx.x < ctas ? __ldcg(p.part_n + threadIdx.x) : 0, s_i);
  for (int o = slices / 2; o > 0; o >>= 1) {
    if (slice < o) {
      s_p[threadIdx.x] += s_p[threadIdx.x + o * width];
      s_c[threadIdx.x] += s_c[threadIdx.x + o * width];
    }
    __syncthreads();
  }
  float weighted = 0.0f;
  if (slice == 0 && e < p.E) {
    p.prob_sum[e] = s_p[e];
    p.counts[e] = s_c[e];
    weighted = s_p[e] * static_cast<float>(s_c[e]);
  }
  weighted = block_sum(weighted, s_f);
  if (threadIdx.x == 0) put_losses(p, weighted, z, n);
}

template <typename S, int L, int V>
__global__ void __launch_bounds__(RT_THREADS) k_route_bwd(const RouteParams p) {
  constexpr int G = RT_THREADS / L;
  const int l = threadIdx.x % L, group = threadIdx.x / L;
  const int E = p.E, k = p.k;
  const float n = fmaxf(static_cast<float>(__ldg(p.counts + E)), 1.0f);
  const float db = p.dlosses != nullptr ? __ldg(p.dlosses) : 0.0f;
  const float dz = p.dlosses != nullptr ? __ldg(p.dlosses + 1) : 0.0f;
  const float unit = db * (static_cast<float>(E) / static_cast<float>(k)) / n / n;
  float c[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = l + L * i;
    c[i] = e < E ? unit * static_cast<float>(__ldg(p.counts + e)) : 0.0f;
    if (e < E && p.dprob_sum != nullptr) c[i] += __ldg(p.dprob_sum + e);
  }
  const S* logits = static_cast<const S*>(p.logits);
  S* dlogits = static_cast<S*>(p.dlogits);
  const int64_t slots = p.T * k;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * G; t0 < p.T; t0 += static_cast<int64_t>(gridDim.x) * G) {
    const int64_t t = t0 + group;
    const bool in = t < p.T;
    const float lse = in ? __ldg(p.lse + t) : -INFINITY;
    const bool on = !(lse == -INFINITY);      // the forward leaves -inf where a token takes no part
    float pr[V];
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      pr[i] = on && l + L * i < E ? expf(load_logit(logits + t * E + l + L * i) - lse) : 0.0f;
      dot += pr[i] * c[i];
    }
    dot = group_sum<L>(dot);
    float gd = 0.0f, g = 0.0f;                // lane j has choice j
    int at = -1;
    if (on && l < k && p.dgates != nullptr) {
      const int64_t slot = t * k + l;
      const int e = __ldg(p.experts + slot);
      g = __ldg(p.gates + slot);
      int64_t from = slot;
      if (p.row_of_slot != nullptr) from = __ldg(p.row_of_slot + slot);
      // a gate of 0 passes nothing on, whatever is in its gradient's place
      if (e >= 0 && e < E && g != 0.0f && from >= 0 && from < slots) {
        at = e;
        gd = g * __ldg(p.dgates + from);
      }
    }
    const float s = group_sum<L>(gd);
    const float add = p.normalize ? gd - g * s : gd;
    const float base = 2.0f * dz / n * lse - dot - (p.normalize ? 0.0f : s);
    float d[V];
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = on ? pr[i] * (c[i] + base) : 0.0f;
    if (p.dgates != nullptr)
      for (int j = 0; j < k; ++j) {
        const float a = __shfl_sync(FULL, add, j, L);
        const int e = __shfl_sync(FULL, at, j, L);
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (e == l + L * i) d[i] += a;
      }
    if (in) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (l + L * i < E) store_logit(dlogits + t * E + l + L * i, d[i]);
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

int lanes_of(int E) { return E <= 4 ? 4 : E <= 8 ? 8 : E <= 16 ? 16 : 32; }

// One CTA up to four tokens per group: a second kernel costs more than they do.
int64_t fwd_ctas(int64_t T, int E) {
  const int64_t groups = RT_THREADS / lanes_of(E);
  return T <= 4 * groups ? 1 : std::min<int64_t>((T + groups - 1) / groups, RT_MAX_CTAS);
}

bool sizes_ok(int64_t T, int E, int k, int dtype) {
  return T >= 0 && E >= 1 && E <= RT_MAX_E && k >= 1 && k <= E && T <= INT32_MAX / k &&
         (dtype == MOE_LOGITS_BF16 || dtype == MOE_LOGITS_F32);
}
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool logits_ok(const void* p, int dtype) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (dtype == MOE_LOGITS_F32 ? 3u : 1u)) == 0;
}

template <bool BWD, typename S, int L, int V>
void launch_one(const RouteParams& p, unsigned grid, cudaStream_t st) {
  if constexpr (BWD)
    k_route_bwd<S, L, V><<<grid, RT_THREADS, 0, st>>>(p);
  else
    k_route_fwd<S, L, V><<<grid, RT_THREADS, (RT_WARPS + 1) * static_cast<size_t>(p.E) * 4, st>>>(p);
}

template <bool BWD, typename S>
void launch_route(const RouteParams& p, unsigned grid, cudaStream_t st) {
  if (p.E <= 4) launch_one<BWD, S, 4, 1>(p, grid, st);
  else if (p.E <= 8) launch_one<BWD, S, 8, 1>(p, grid, st);
  else if (p.E <= 16) launch_one<BWD, S, 16, 1>(p, grid, st);
  else if (p.E <= 32) launch_one<BWD, S, 32, 1>(p, grid, st);
  else if (p.E <= 64) launch_one<BWD, S, 32, 2>(p, grid, st);
  else if (p.E <= 128) launch_one<BWD, S, 32, 4>(p, grid, st);
  else if (p.E <= 256) launch_one<BWD, S, 32, 8>(p, grid, st);
  else if (p.E <= 512) launch_one<BWD, S, 32, 16>(p, grid, st);
  else launch_one<BWD, S, 32, 32>(p, grid, st);
}

}  // namespace
}  // namespace mx

using namespace mx;

extern "C" {

size_t moe_route_workspace_size(int64_t T, int E, int k) {
  if (!sizes_ok(T, E, k, MOE_LOGITS_F32) || k > RT_MAX_K) return 0;
  return static_cast<size_t>(fwd_ctas(T, E)) * (2 * E + 2) * 4;
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
  const int64_t ctas = fwd_ctas(T, E);
  if (ctas > 1) {
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
  p.part_p = static_cast<float*>(workspace);
  p.part_c = reinterpret_cast<int32_t*>(p.part_p + ctas * E);
  p.part_z = reinterpret_cast<float*>(p.part_c + ctas * E);
  p.part_n = reinterpret_cast<int32_t*>(p.part_z + ctas);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (logits_dtype == MOE_LOGITS_F32) launch_route<false, float>(p, static_cast<unsigned>(ctas), st);
  else launch_route<false, uint16_t>(p, static_cast<unsigned>(ctas), st);
  if (cudaGetLastError() != cudaSuccess) return MXFP8_ERR_CUDA;
  if (ctas > 1) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1, 1, 1);
    cfg.blockDim = dim3(RT_FINAL_THREADS, 1, 1);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, k_route_final, p, static_cast<int>(ctas)) != cudaSuccess) return MXFP8_ERR_CUDA;
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
  const int64_t groups = RT_THREADS / lanes_of(E);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>((T + groups - 1) / groups, 8 * sms));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (logits_dtype == MOE_LOGITS_F32) launch_route<true, float>(p, grid, st);
  else launch_route<true, uint16_t>(p, grid, st);
  return cudaGetLastError() == cudaSuccess ? MXFP8_OK : MXFP8_ERR_CUDA;
}

}  // extern "C"

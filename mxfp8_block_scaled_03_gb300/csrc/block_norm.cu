// block_norm.cu -- the junction between two blocks of a decoder, in one pass over the row: RMS norm of
// the block's output (post-norm), its gate, the scaled residual, and the RMS norm in front of the next
// block (pre-norm); forward and backward.
//
//   yh = y / rms(y), z = yh * w_post (z = y without the post-norm)
//   r' = res_scale * r + gate * z,   rh = r' / rms(r'),   n = rh * w_pre
// and for the gradients dn of n and dr' of r':
//   g  = dr' + (a - rh mean(a rh)) / rms(r'),  a = dn * w_pre        (the whole gradient of r')
//   dr = res_scale * g;   dz = gate * g;   dgate = sum of g * z over the gate's broadcast axis
//   dy = (b - yh mean(b yh)) / rms(y),  b = dz * w_post  (dz without the post-norm)
//   dw_post = sum over rows of dz * yh,   dw_pre = sum over rows of dn * rh
// rms(v) = sqrt(mean(v^2) + eps).  All of it in 32 bits; what is stored as bf16 is rounded once.
//
// What bounds it: HBM (forward: y, r in, r', n out, 8 bytes per element with a bf16 residual; backward:
// dn, dr', y, r' in, dy, dr out, 12 bytes).  A row needs two sums over its length, the second of which
// depends on the first, so a row costs two exchanges between its threads; to keep memory busy
// meanwhile, every thread copies its own 16-byte pieces of the next rows into shared memory with
// cp.async (no barrier: nobody else reads them) while it works on this one.  CTAs are persistent, so
// weights stay in registers and the backward's column sums accumulate there; a second kernel adds the
// CTAs' sums in a fixed order.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>

#include "mx_device.cuh"
#include "mx_internal.h"
#include "mxfp8moe.h"

namespace mx {
namespace {

constexpr int BN_THREADS = 512;          // most threads of a CTA
constexpr int BN_MAX_H = 8192;           // two vectors of 8 values per thread
constexpr int BN_MAX_STAGES = 4;
constexpr int COLS_THREADS = 1024;       // column sums: 32 columns x 32 shares of the CTAs

struct NormParams {
  const void *y, *res, *dn, *dres_out;   // forward: y, res; backward: y, res_out (as res), dn, dres_out
  const float *w_post, *gate, *w_pre;
  void *res_out, *n, *dy, *dres;
  float* stats;                          // [2, T]: 1 / rms of y and of r'
  float *dw_post, *dgate, *dw_pre;
  float* part;                           // backward: [gridDim.x][2][H] column sums (one CTA: unused)
  int64_t T;
  int H, nv;                             // nv = H / 8 vectors per row
  int tpr, groups;                       // threads per row (a multiple of 32), rows per CTA at a time
  int stages;
  int gate_kind, post;
  int wide;                              // the residual outputs are 32-byte aligned
  float res_scale, eps;
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest `pending` groups have arrived (pending is at most BN_MAX_STAGES - 1).
__device__ __forceinline__ void cp_async_wait(int pending) {
  switch (pending) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
  }
}

// Gradients of column c from its finished sum: k = 0: S (see the backward), k = 1: dw_pre.
__device__ __forceinline__ void put_columns(const NormParams& p, int k, int c, float v) {
  if (k == 1) {
    if (p.dw_pre != nullptr) p.dw_pre[c] = v;
    return;
  }
  const bool channel = p.gate_kind == RESIDUAL_GATE_CHANNEL;
  if (p.dw_post != nullptr) p.dw_post[c] = channel ? v * __ldg(p.gate + c) : v;
  if (channel && p.dgate != nullptr) p.dgate[c] = p.w_post != nullptr ? v * __ldg(p.w_post + c) : v;
}

// Eight values as four pairs of floats (the SM's f32x2 arithmetic: one instruction per pair), from 16
// bytes of bf16 or two 16-byte halves of float, `stride` pieces apart.
using Vec8 = uint64_t[4];
__device__ __forceinline__ uint64_t f2_splat(float v) { return f2_pack(v, v); }
__device__ __forceinline__ void unpack(const uint4* p, Vec8& v, int, uint16_t) {
  const uint4 w = *p;
  v[0] = f2_pack(bf16_lo(w.x), bf16_hi(w.x));
  v[1] = f2_pack(bf16_lo(w.y), bf16_hi(w.y));
  v[2] = f2_pack(bf16_lo(w.z), bf16_hi(w.z));
  v[3] = f2_pack(bf16_lo(w.w), bf16_hi(w.w));
}
__device__ __forceinline__ void unpack(const uint4* p, Vec8& v, int stride, float) {
  const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(p), b = *reinterpret_cast<const ulonglong2*>(p + stride);
  v[0] = a.x;
  v[1] = a.y;
  v[2] = b.x;
  v[3] = b.y;
}
__device__ __forceinline__ uint32_t to_bf16x2(uint64_t v) { return pack_bf16x2(f2_lo(v), f2_hi(v)); }
__device__ __forceinline__ void store8(uint16_t* dst, const Vec8& v, int) {
  __stcs(reinterpret_cast<uint4*>(dst), make_uint4(to_bf16x2(v[0]), to_bf16x2(v[1]), to_bf16x2(v[2]), to_bf16x2(v[3])));
}
// Floats: one 32-byte store, a whole sector, where the alignment allows (two 16-byte stores of a warp each
// touch every sector by half).
__device__ __forceinline__ void store8(float* dst, const Vec8& v, int wide) {
  const uint4 a = make_uint4(static_cast<uint32_t>(v[0]), static_cast<uint32_t>(v[0] >> 32),
                             static_cast<uint32_t>(v[1]), static_cast<uint32_t>(v[1] >> 32));
  const uint4 b = make_uint4(static_cast<uint32_t>(v[2]), static_cast<uint32_t>(v[2] >> 32),
                             static_cast<uint32_t>(v[3]), static_cast<uint32_t>(v[3] >> 32));
  if (wide) {
    st_global_32B_cs(dst, a, b);
  } else {
    __stcs(reinterpret_cast<uint4*>(dst), a);
    __stcs(reinterpret_cast<uint4*>(dst) + 1, b);
  }
}
// Eight weights, or ones where there are none.
__device__ __forceinline__ void load8(const float* src, Vec8& v) {
  if (src != nullptr) {
    unpack(reinterpret_cast<const uint4*>(src), v, 1, 0.0f);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2_splat(1.0f);
  }
}

// Sum over the threads of a row: shuffles inside a warp, shared memory between the row's warps (two
// buffers in turn: one barrier per sum).  The order of the additions is fixed.
struct RowSum {
  float* slots;   // [2][16 warps], with two sums at a time [2][2][16 warps]
  int warp0, warps, barrier, tpr;
  int buf = 0;
  __device__ __forceinline__ float operator()(uint64_t v) {
    float a = f2_lo(v) + f2_hi(v);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, d);
    if (warps == 1) return a;
    float* s = slots + buf * (BN_THREADS / 32) + warp0;
    buf ^= 1;
    const int lane = threadIdx.x & 31;
    if (lane == 0) s[(threadIdx.x >> 5) - warp0] = a;
    asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(tpr) : "memory");
    a = lane < warps ? s[lane] : 0.0f;   // at most 16 warps
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, d);
    return __shfl_sync(0xFFFFFFFFu, a, 0);
  }
  // two sums with one barrier
  __device__ __forceinline__ float2 operator()(uint64_t v, uint64_t w) {
    float a = f2_lo(v) + f2_hi(v), b = f2_lo(w) + f2_hi(w);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
      a += __shfl_xor_sync(0xFFFFFFFFu, a, d);
      b += __shfl_xor_sync(0xFFFFFFFFu, b, d);
    }
    if (warps == 1) return make_float2(a, b);
    float* s = slots + buf * (BN_THREADS / 32) + warp0;
    float* t = s + 2 * (BN_THREADS / 32);
    buf ^= 1;
    const int lane = threadIdx.x & 31;
    if (lane == 0) {
      s[(threadIdx.x >> 5) - warp0] = a;
      t[(threadIdx.x >> 5) - warp0] = b;
    }
    asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(tpr) : "memory");
    // lanes 0-15 add the first sum's parts, lanes 16-31 the second's
    a = (lane & 15) < warps ? (lane < 16 ? s : t)[lane & 15] : 0.0f;
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, d);
    return make_float2(__shfl_sync(0xFFFFFFFFu, a, 0), __shfl_sync(0xFFFFFFFFu, a, 16));
  }
};

// Where a thread stands: its row group, its place in the row, and the ring of its prefetched pieces.
// A stage holds, per vector, PIECES blocks of one 16-byte piece per thread.  A bf16 array takes one block:
// a thread copies and reads its own piece.  A float array takes two: a warp copies its 1 KB in two contiguous
// halves (32 bytes per lane in one piece would fetch every sector twice), and a lane reads pieces 2l, 2l + 1.
template <int V, int PIECES>
struct Lane {
  int group, t, tpr, nv;
  uint4* ring;
  __device__ __forceinline__ uint4* block(int stage, int v, int i) const {
    return ring + ((stage * V + v) * PIECES + i) * blockDim.x;
  }
  // from array[o ..], o being where the row starts
  __device__ __forceinline__ void copy(const uint16_t* array, int64_t o, int stage, int v, int i) const {
    const int j = t + v * tpr;
    if (j < nv) cp_async16(block(stage, v, i) + threadIdx.x, array + o + j * 8);
  }
  __device__ __forceinline__ void copy(const float* array, int64_t o, int stage, int v, int i) const {
    const int lane = threadIdx.x & 31;
    uint4* dst = block(stage, v, i) + (threadIdx.x - lane) * 2;
    const int j = (t - lane + v * tpr) * 2 + lane;   // in units of four floats
    if (j < 2 * nv) cp_async16(dst + lane, array + o + j * 4);
    if (j + 32 < 2 * nv) cp_async16(dst + 32 + lane, array + o + (j + 32) * 4);
  }
  __device__ __forceinline__ void read(int stage, int v, int i, Vec8& out, uint16_t) const {
    unpack(block(stage, v, i) + threadIdx.x, out, 0, uint16_t{});
  }
  __device__ __forceinline__ void read(int stage, int v, int i, Vec8& out, float) const {
    unpack(block(stage, v, i) + threadIdx.x * 2, out, 1, 0.0f);
  }
};

template <typename RT, int V>
__global__ void __launch_bounds__(BN_THREADS, V == 1 ? 2 : 1) k_residual_norm_fwd(const NormParams p) {
  constexpr int RP = sizeof(RT) / 2;        // 16-byte pieces of 8 residual values
  constexpr int PIECES = 1 + RP;
  extern __shared__ uint4 ring[];
  __shared__ float s_sum[2 * BN_THREADS / 32];
  Lane<V, PIECES> me{static_cast<int>(threadIdx.x) / p.tpr, static_cast<int>(threadIdx.x) % p.tpr, p.tpr, p.nv, ring};
  RowSum row_sum{s_sum, me.group * (p.tpr / 32), p.tpr / 32, 1 + me.group, p.tpr};
  const int64_t step = static_cast<int64_t>(gridDim.x) * p.groups;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * p.groups + me.group;
  const uint16_t* y = static_cast<const uint16_t*>(p.y);
  const RT* res = static_cast<const RT*>(p.res);
  const float inv_h = 1.0f / static_cast<float>(p.H);
  bool in[V];
#pragma unroll
  for (int v = 0; v < V; ++v) in[v] = me.t + v * p.tpr < p.nv;

  auto fetch = [&](int64_t row, int stage) {
    if (RP == 2) __syncwarp();   // the warp has read what the stage held
    if (row < p.T) {
      const int64_t o = row * p.H;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        me.copy(y, o, stage, v, 0);
        me.copy(res, o, stage, v, 1);
      }
    }
    cp_async_commit();
  };
  // post-norm weight times channel gate, and pre-norm weight
  Vec8 wa[V], wb[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (me.t + v * p.tpr) * 8;
    Vec8 g;
    load8(in[v] && p.w_post != nullptr ? p.w_post + c : nullptr, wa[v]);
    load8(in[v] && p.gate_kind == RESIDUAL_GATE_CHANNEL ? p.gate + c : nullptr, g);
    load8(in[v] && p.w_pre != nullptr ? p.w_pre + c : nullptr, wb[v]);
#pragma unroll
    for (int i = 0; i < 4; ++i) wa[v][i] = f2_mul(wa[v][i], g[i]);
  }
  for (int s = 0; s + 1 < p.stages; ++s) fetch(first + s * step, s);

  // the row's token gate, read one row ahead
  const float* tgate = p.gate_kind == RESIDUAL_GATE_TOKEN ? p.gate : nullptr;
  float next_tg = tgate != nullptr && first < p.T ? __ldg(tgate + first) : 1.0f;
  const uint64_t scale = f2_splat(p.res_scale);
  int stage = 0;
  for (int64_t row = first; row < p.T; row += step) {
    fetch(row + (p.stages - 1) * step, stage == 0 ? p.stages - 1 : stage - 1);
    const float tg = next_tg;
    if (tgate != nullptr && row + step < p.T) next_tg = __ldg(tgate + row + step);
    cp_async_wait(p.stages - 1);
    if (RP == 2) __syncwarp();
    Vec8 z[V], r[V];
    uint64_t ss = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) z[v][i] = r[v][i] = 0;
      if (in[v]) {
        me.read(stage, v, 0, z[v], uint16_t{});
        me.read(stage, v, 1, r[v], RT{});
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) ss = f2_fma(z[v][i], z[v][i], ss);
    }
    const float rs1 = p.post ? rsqrtf(fmaf(row_sum(ss), inv_h, p.eps)) : 1.0f;
    const uint64_t zs = f2_splat(rs1 * tg);
    ss = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r[v][i] = f2_fma(f2_mul(z[v][i], zs), wa[v][i], f2_mul(r[v][i], scale));
        ss = f2_fma(r[v][i], r[v][i], ss);
      }
      if (in[v]) store8(static_cast<RT*>(p.res_out) + row * p.H + (me.t + v * p.tpr) * 8, r[v], p.wide);
    }
    const float rs2 = rsqrtf(fmaf(row_sum(ss), inv_h, p.eps));
    const uint64_t ns = f2_splat(rs2);
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) r[v][i] = f2_mul(f2_mul(r[v][i], ns), wb[v][i]);
      if (in[v]) store8(static_cast<uint16_t*>(p.n) + row * p.H + (me.t + v * p.tpr) * 8, r[v], 0);
    }
    if (me.t == 0) {
      p.stats[row] = rs1;
      p.stats[p.T + row] = rs2;
    }
    if (++stage == p.stages) stage = 0;
  }
}

// With S = sum over rows of (token gate) g yh per column: dw_post = (channel gate) S and
// dgate = w_post S (channel), and a token's dgate is the row sum of g yh w_post that the norm's gradient
// needs anyway; so one column sum serves both, next to that of dw_pre.  Thread t of a group owns columns
// 8 (t + v tpr) ..; the groups of a CTA are added in order through shared memory at the end (the ring's space).
template <typename RT, int V>
__global__ void __launch_bounds__(BN_THREADS, 1) k_residual_norm_bwd(const NormParams p) {
  constexpr int RP = sizeof(RT) / 2;
  constexpr int PIECES = 2 + 2 * RP;        // dn, y, r', dr'
  extern __shared__ uint4 ring[];
  __shared__ float s_sum[4 * BN_THREADS / 32];
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Lane<V, PIECES> me{static_cast<int>(threadIdx.x) / p.tpr, static_cast<int>(threadIdx.x) % p.tpr, p.tpr, p.nv, ring};
  RowSum row_sum{s_sum, me.group * (p.tpr / 32), p.tpr / 32, 1 + me.group, p.tpr};
  const int64_t step = static_cast<int64_t>(gridDim.x) * p.groups;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * p.groups + me.group;
  const uint16_t *dn = static_cast<const uint16_t*>(p.dn), *y = static_cast<const uint16_t*>(p.y);
  const RT *res = static_cast<const RT*>(p.res), *dro = static_cast<const RT*>(p.dres_out);
  const float inv_h = 1.0f / static_cast<float>(p.H);
  bool in[V];
#pragma unroll
  for (int v = 0; v < V; ++v) in[v] = me.t + v * p.tpr < p.nv;

  auto fetch = [&](int64_t row, int stage) {
    if (RP == 2) __syncwarp();   // the warp has read what the stage held
    if (row < p.T) {
      const int64_t o = row * p.H;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        me.copy(dn, o, stage, v, 0);
        me.copy(y, o, stage, v, 1);
        me.copy(res, o, stage, v, 2);
        if (dro != nullptr) me.copy(dro, o, stage, v, 2 + RP);
      }
    }
    cp_async_commit();
  };
  Vec8 wa[V], wb[V];       // post-norm weight times channel gate, pre-norm weight
  Vec8 sa[V], sb[V];       // column sums: S, dw_pre
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (me.t + v * p.tpr) * 8;
    Vec8 g;
    load8(in[v] && p.w_post != nullptr ? p.w_post + c : nullptr, wa[v]);
    load8(in[v] && p.gate_kind == RESIDUAL_GATE_CHANNEL ? p.gate + c : nullptr, g);
    load8(in[v] && p.w_pre != nullptr ? p.w_pre + c : nullptr, wb[v]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      wa[v][i] = f2_mul(wa[v][i], g[i]);
      sa[v][i] = sb[v][i] = 0;
    }
  }
  for (int s = 0; s + 1 < p.stages; ++s) fetch(first + s * step, s);

  // the rows' scalars, read a row ahead of their use
  const float* tgate = p.gate_kind == RESIDUAL_GATE_TOKEN ? p.gate : nullptr;
  struct Scalars {
    float rs1, rs2, tg;
  };
  auto scalars = [&](int64_t row) {
    Scalars q{1.0f, 1.0f, 1.0f};
    if (row >= p.T) return q;
    if (p.post) q.rs1 = __ldg(p.stats + row);
    q.rs2 = __ldg(p.stats + p.T + row);
    if (tgate != nullptr) q.tg = __ldg(tgate + row);
    return q;
  };
  // First half of a row: a = dn w_pre and rh, the column sum of dw_pre, this thread's share of sum(a rh).
  Vec8 a[V], rh[V];
  auto first_half = [&](int stage, float rs2, bool live) {
    const uint64_t k2 = f2_splat(rs2);
    uint64_t s1 = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) a[v][i] = rh[v][i] = 0;
      if (in[v] && live) {
        me.read(stage, v, 0, a[v], uint16_t{});
        me.read(stage, v, 2, rh[v], RT{});
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        rh[v][i] = f2_mul(rh[v][i], k2);
        sb[v][i] = f2_fma(a[v][i], rh[v][i], sb[v][i]);
        a[v][i] = f2_mul(a[v][i], wb[v][i]);
        s1 = f2_fma(a[v][i], rh[v][i], s1);
      }
    }
    return s1;
  };
  // The second half of a row and the first half of the next run between two barriers, so that a row costs
  // one exchange between its warps instead of two (16384 x 4096, bf16, column sums included: 162 -> 150 us).  With two
  // vectors per thread the registers do not hold both (8192 x 8192: 190 -> 272 us): there the halves follow each other.
  const uint64_t scale = f2_splat(p.res_scale);
  Scalars cur = scalars(first), next = scalars(first + step);
  cp_async_wait(p.stages - 2);
  __syncwarp();
  float m1 = first < p.T ? row_sum(first_half(0, cur.rs2, true)) * -inv_h : 0.0f;
  int stage = 0;
  for (int64_t row = first; row < p.T; row += step) {
    fetch(row + (p.stages - 1) * step, stage == 0 ? p.stages - 1 : stage - 1);
    const Scalars after = scalars(row + 2 * step);
    const uint64_t k1 = f2_splat(cur.rs1), k2 = f2_splat(cur.rs2), kt = f2_splat(cur.tg), km = f2_splat(m1);
    Vec8 b[V], yh[V];
    uint64_t s2 = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      Vec8 g;
#pragma unroll
      for (int i = 0; i < 4; ++i) g[i] = yh[v][i] = 0;
      if (in[v]) {
        me.read(stage, v, 1, yh[v], uint16_t{});
        if (dro != nullptr) me.read(stage, v, 2 + RP, g, RT{});
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        g[i] = f2_fma(f2_fma(rh[v][i], km, a[v][i]), k2, g[i]);
        yh[v][i] = f2_mul(yh[v][i], k1);
        const uint64_t gy = f2_mul(g[i], yh[v][i]);
        sa[v][i] = f2_fma(gy, kt, sa[v][i]);
        b[v][i] = f2_mul(g[i], wa[v][i]);
        s2 = f2_fma(gy, wa[v][i], s2);
        g[i] = f2_mul(g[i], scale);
      }
      if (in[v]) store8(static_cast<RT*>(p.dres) + row * p.H + (me.t + v * p.tpr) * 8, g, p.wide);
    }
    if (++stage == p.stages) stage = 0;
    cp_async_wait(p.stages - 2);
    if (RP == 2) __syncwarp();
    const bool more = row + step < p.T;
    float2 sums;
    if (V == 1) {
      sums = row_sum(s2, first_half(stage, next.rs2, more));
      m1 = sums.y * -inv_h;
    } else {
      sums.x = row_sum(s2);
    }
    const uint64_t m2 = f2_splat(p.post ? -sums.x * inv_h : 0.0f), ky = f2_splat(cur.rs1 * cur.tg);
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) b[v][i] = f2_mul(f2_fma(yh[v][i], m2, b[v][i]), ky);
      if (in[v]) store8(static_cast<uint16_t*>(p.dy) + row * p.H + (me.t + v * p.tpr) * 8, b[v], 0);
    }
    if (V > 1) m1 = row_sum(first_half(stage, next.rs2, more)) * -inv_h;
    if (me.t == 0 && tgate != nullptr && p.dgate != nullptr) p.dgate[row] = sums.x;
    cur = next;
    next = after;
  }

  // the groups' column sums, added in order; then to the CTA's place (or, alone, to the results)
  cp_async_wait(0);
  __syncthreads();
  float2* sums = reinterpret_cast<float2*>(ring);   // [2][H / 2]
  for (int g = 0; g < p.groups; ++g) {
    if (me.group == g) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (!in[v]) continue;
        float2* s = sums + (me.t + v * p.tpr) * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = s[i], z = s[p.H / 2 + i];
          s[i] = make_float2(f2_lo(sa[v][i]) + (g ? x.x : 0.0f), f2_hi(sa[v][i]) + (g ? x.y : 0.0f));
          s[p.H / 2 + i] = make_float2(f2_lo(sb[v][i]) + (g ? z.x : 0.0f), f2_hi(sb[v][i]) + (g ? z.y : 0.0f));
        }
      }
    }
    __syncthreads();
  }
  const float* flat = reinterpret_cast<const float*>(sums);
  for (int c = threadIdx.x; c < p.H; c += static_cast<int>(blockDim.x)) {
    if (gridDim.x == 1) {
      put_columns(p, 0, c, flat[c]);
      put_columns(p, 1, c, flat[p.H + c]);
    } else {
      float* part = p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.H;
      part[c] = flat[c];
      part[p.H + c] = flat[p.H + c];
    }
  }
}

// Adds the CTAs' column sums part[.][k][c].  A CTA takes 32 columns of one k; its warps take equal shares of the
// CTAs, added in order: five trips to the L2 at once instead of 19 in turn (16384 x 4096, the backward as a whole:
// 150 us, with 8 warps 152; 1531 x 2048: 16.4 and 18.2).
__global__ void __launch_bounds__(COLS_THREADS) k_norm_columns(const NormParams p, int ctas) {
  __shared__ float s[COLS_THREADS / 32][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int k = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const int per = (ctas + COLS_THREADS / 32 - 1) / (COLS_THREADS / 32);
  float v = 0.0f;
  if (c < p.H) {
    const int end = min(ctas, (warp + 1) * per);
#pragma unroll 8
    for (int i = warp * per; i < end; ++i) v += __ldcg(p.part + (static_cast<int64_t>(i) * 2 + k) * p.H + c);
  }
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < p.H) {
    for (int w = 1; w < COLS_THREADS / 32; ++w) v += s[w][lane];
    put_columns(p, k, c, v);
  }
}

// ---- host side -------------------------------------------------------------------------------

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr size_t BN_SMEM = 224 * 1024;   // of one SM
struct NormShape {
  int v, tpr, groups, threads, stages, per_sm;
  size_t smem;
};
// pieces: 16-byte pieces per vector of 8 values that a stage holds.  The forward with one vector per thread
// has two CTAs per SM, everything else one.
NormShape norm_shape(int H, int pieces, bool bwd, size_t least) {
  NormShape s{};
  const int nv = H / 8;
  // two vectors per thread beyond 2048 columns: fewer warps to exchange sums with (forward, 16384 x 4096: 101 ->
  // 91 us); the backward's registers hold only one (150 against 174 us), so beyond 4096 columns, where it needs two, it
  // runs at 50 to 63% of the copy (13000 x 5120: 238 us, 8192 x 8192: 190)
  s.v = nv <= (bwd ? BN_THREADS : BN_THREADS / 2) ? 1 : 2;
  s.tpr = ((nv + s.v - 1) / s.v + 31) / 32 * 32;
  s.groups = std::max(1, BN_THREADS / s.tpr);
  if (s.tpr > 32) s.groups = std::min(s.groups, 15);   // one hardware barrier per group
  s.threads = s.tpr * s.groups;
  s.per_sm = !bwd && s.v == 1 ? 2 : 1;
  const size_t budget = BN_SMEM / s.per_sm;
  const size_t stage = static_cast<size_t>(s.v) * pieces * s.threads * 16;
  s.stages = static_cast<int>(std::min<size_t>(BN_MAX_STAGES, budget / stage));
  s.smem = std::max(stage * s.stages, least);
  return s;
}

struct NormDevice {
  int sms;
};
// Shared-memory limits of the kernels, once per device; false on failure.
bool norm_device(NormDevice* out) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> sms[kMaxDevices] = {};
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
  if ((n = sms[dev].load()) <= 0) {
    const void* fwd[] = {reinterpret_cast<const void*>(k_residual_norm_fwd<uint16_t, 1>),
                         reinterpret_cast<const void*>(k_residual_norm_fwd<uint16_t, 2>),
                         reinterpret_cast<const void*>(k_residual_norm_fwd<float, 1>),
                         reinterpret_cast<const void*>(k_residual_norm_fwd<float, 2>)};
    const void* bwd[] = {reinterpret_cast<const void*>(k_residual_norm_bwd<uint16_t, 1>),
                         reinterpret_cast<const void*>(k_residual_norm_bwd<uint16_t, 2>),
                         reinterpret_cast<const void*>(k_residual_norm_bwd<float, 1>),
                         reinterpret_cast<const void*>(k_residual_norm_bwd<float, 2>)};
    for (int i = 0; i < 4; ++i)
      if (cudaFuncSetAttribute(fwd[i], cudaFuncAttributeMaxDynamicSharedMemorySize, BN_SMEM) != cudaSuccess ||
          cudaFuncSetAttribute(bwd[i], cudaFuncAttributeMaxDynamicSharedMemorySize, BN_SMEM) != cudaSuccess)
        return false;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return false;
    sms[dev].store(n);
  }
  out->sms = n;
  return true;
}

// CTAs of the backward (the workspace holds their column sums; the same on every device).
constexpr int BN_MAX_CTAS = 160;

bool sizes_ok(int64_t T, int64_t H, int res_dtype, int gate_kind, int post_norm) {
  return T >= 0 && H > 0 && (res_dtype == RESIDUAL_BF16 || res_dtype == RESIDUAL_F32) &&
         (gate_kind == RESIDUAL_GATE_NONE || gate_kind == RESIDUAL_GATE_CHANNEL || gate_kind == RESIDUAL_GATE_TOKEN) &&
         (post_norm == 0 || post_norm == 1);
}

}  // namespace
}  // namespace mx

using namespace mx;

extern "C" {

int residual_norm_fwd(const void* y, const void* res, const float* w_post, const float* gate, const float* w_pre,
                      int64_t T, int64_t H, int res_dtype, int gate_kind, int post_norm, float res_scale, float eps,
                      void* res_out, void* n, float* stats, void* stream) {
  if (!sizes_ok(T, H, res_dtype, gate_kind, post_norm)) return MXFP8_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || (gate != nullptr) != (gate_kind != RESIDUAL_GATE_NONE) || (w_post != nullptr && !post_norm))
    return MXFP8_ERR_INVALID_ARG;
  if (H % 8 != 0 || H > BN_MAX_H) return MXFP8_ERR_UNSUPPORTED;
  if (T == 0) return MXFP8_OK;
  for (const void* q : {y, res, static_cast<const void*>(res_out), static_cast<const void*>(n)})
    if (q == nullptr || !aligned16(q)) return MXFP8_ERR_INVALID_ARG;
  if (stats == nullptr || !aligned16(w_post) || !aligned16(w_pre) || (reinterpret_cast<uintptr_t>(stats) & 3u) != 0 ||
      (gate_kind == RESIDUAL_GATE_CHANNEL ? !aligned16(gate) : (reinterpret_cast<uintptr_t>(gate) & 3u) != 0))
    return MXFP8_ERR_INVALID_ARG;
  NormDevice dev;
  if (!norm_device(&dev)) return MXFP8_ERR_CUDA;
  const bool f32 = res_dtype == RESIDUAL_F32;
  const NormShape s = norm_shape(static_cast<int>(H), f32 ? 3 : 2, false, 0);
  NormParams p{};
  p.y = y;
  p.res = res;
  p.w_post = w_post;
  p.gate = gate;
  p.w_pre = w_pre;
  p.res_out = res_out;
  p.n = n;
  p.stats = stats;
  p.T = T;
  p.H = static_cast<int>(H);
  p.nv = p.H / 8;
  p.tpr = s.tpr;
  p.groups = s.groups;
  p.stages = s.stages;
  p.gate_kind = gate_kind;
  p.post = post_norm;
  p.wide = (reinterpret_cast<uintptr_t>(res_out) & 31u) == 0;
  p.res_scale = res_scale;
  p.eps = eps;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>((T + s.groups - 1) / s.groups, s.per_sm * dev.sms));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (f32) {
    if (s.v == 1) k_residual_norm_fwd<float, 1><<<grid, s.threads, s.smem, st>>>(p);
    else k_residual_norm_fwd<float, 2><<<grid, s.threads, s.smem, st>>>(p);
  } else {
    if (s.v == 1) k_residual_norm_fwd<uint16_t, 1><<<grid, s.threads, s.smem, st>>>(p);
    else k_residual_norm_fwd<uint16_t, 2><<<grid, s.threads, s.smem, st>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? MXFP8_OK : MXFP8_ERR_CUDA;
}

size_t residual_norm_bwd_workspace_size(int64_t T, int64_t H) {
  if (T < 0 || H <= 0 || H > BN_MAX_H) return 0;
  return static_cast<size_t>(std::min<int64_t>(T, BN_MAX_CTAS)) * 2 * H * sizeof(float);
}

int residual_norm_bwd(const void* dn, const void* dres_out, const void* y, const void* res_out, const float* stats,
                      const float* w_post, const float* gate, const float* w_pre, int64_t T, int64_t H, int res_dtype,
                      int gate_kind, int post_norm, float res_scale, void* dy, void* dres, float* dw_post,
                      float* dgate, float* dw_pre, void* workspace, size_t workspace_bytes, void* stream) {
  if (!sizes_ok(T, H, res_dtype, gate_kind, post_norm)) return MXFP8_ERR_INVALID_ARG;
  if ((gate != nullptr) != (gate_kind != RESIDUAL_GATE_NONE) || (w_post != nullptr && !post_norm))
    return MXFP8_ERR_INVALID_ARG;
  // a gradient is asked for only where the weight exists
  if ((dw_post != nullptr && w_post == nullptr) || (dgate != nullptr && gate == nullptr) ||
      (dw_pre != nullptr && w_pre == nullptr))
    return MXFP8_ERR_INVALID_ARG;
  if (H % 8 != 0 || H > BN_MAX_H) return MXFP8_ERR_UNSUPPORTED;
  for (const void* q : {static_cast<const void*>(dw_post), static_cast<const void*>(dgate),
                        static_cast<const void*>(dw_pre), static_cast<const void*>(w_post),
                        static_cast<const void*>(w_pre), dres_out})
    if (!aligned16(q)) return MXFP8_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {   // sums over no rows
    const size_t row = static_cast<size_t>(H) * sizeof(float);
    if ((dw_post != nullptr && cudaMemsetAsync(dw_post, 0, row, st) != cudaSuccess) ||
        (dw_pre != nullptr && cudaMemsetAsync(dw_pre, 0, row, st) != cudaSuccess) ||
        (dgate != nullptr && gate_kind == RESIDUAL_GATE_CHANNEL && cudaMemsetAsync(dgate, 0, row, st) != cudaSuccess))
      return MXFP8_ERR_CUDA;
    return MXFP8_OK;
  }
  for (const void* q : {dn, y, res_out, static_cast<const void*>(dy), static_cast<const void*>(dres)})
    if (q == nullptr || !aligned16(q)) return MXFP8_ERR_INVALID_ARG;
  if (stats == nullptr || (reinterpret_cast<uintptr_t>(stats) & 3u) != 0 ||
      (gate_kind == RESIDUAL_GATE_CHANNEL ? !aligned16(gate) : (reinterpret_cast<uintptr_t>(gate) & 3u) != 0))
    return MXFP8_ERR_INVALID_ARG;
  NormDevice dev;
  if (!norm_device(&dev)) return MXFP8_ERR_CUDA;
  const bool f32 = res_dtype == RESIDUAL_F32;
  const NormShape s = norm_shape(static_cast<int>(H), f32 ? 6 : 4, true, static_cast<size_t>(H) * 8);
  const int64_t ctas = std::min<int64_t>((T + s.groups - 1) / s.groups, std::min(dev.sms, BN_MAX_CTAS));
  if (ctas > 1) {
    if (workspace == nullptr || !aligned16(workspace)) return MXFP8_ERR_INVALID_ARG;
    if (workspace_bytes < static_cast<size_t>(ctas) * 2 * H * sizeof(float)) return MXFP8_ERR_WORKSPACE;
  }
  NormParams p{};
  p.y = y;
  p.res = res_out;
  p.dn = dn;
  p.dres_out = dres_out;
  p.w_post = w_post;
  p.gate = gate;
  p.w_pre = w_pre;
  p.dy = dy;
  p.dres = dres;
  p.stats = const_cast<float*>(stats);
  p.dw_post = dw_post;
  p.dgate = dgate;
  p.dw_pre = dw_pre;
  p.part = static_cast<float*>(workspace);
  p.T = T;
  p.H = static_cast<int>(H);
  p.nv = p.H / 8;
  p.tpr = s.tpr;
  p.groups = s.groups;
  p.stages = s.stages;
  p.gate_kind = gate_kind;
  p.post = post_norm;
  p.wide = (reinterpret_cast<uintptr_t>(dres) & 31u) == 0;
  p.res_scale = res_scale;
  const unsigned grid = static_cast<unsigned>(ctas);
  if (f32) {
    if (s.v == 1) k_residual_norm_bwd<float, 1><<<grid, s.threads, s.smem, st>>>(p);
    else k_residual_norm_bwd<float, 2><<<grid, s.threads, s.smem, st>>>(p);
  } else {
    if (s.v == 1) k_residual_norm_bwd<uint16_t, 1><<<grid, s.threads, s.smem, st>>>(p);
    else k_residual_norm_bwd<uint16_t, 2><<<grid, s.threads, s.smem, st>>>(p);
  }
  if (cudaGetLastError() != cudaSuccess) return MXFP8_ERR_CUDA;
  float* cols = gate_kind == RESIDUAL_GATE_CHANNEL ? dgate : nullptr;
  if (ctas > 1 && (dw_post != nullptr || cols != nullptr || dw_pre != nullptr)) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((p.H + 31) / 32, 2, 1);
    cfg.blockDim = dim3(COLS_THREADS, 1, 1);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, k_norm_columns, p, static_cast<int>(ctas)) != cudaSuccess) return MXFP8_ERR_CUDA;
  }
  return MXFP8_OK;
}

}  // extern "C"

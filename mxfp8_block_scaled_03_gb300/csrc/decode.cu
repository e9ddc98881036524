// decode.cu -- the expert MLP and plain linears for a few tokens (decode steps): a whole MoE layer
// in two kernels, and y = x W^T for a few rows of x, from the MXFP8 and NVFP4 weights the grouped
// GEMMs use (same codes, same tensor-core scale layout).
//
//   moe_decode_fwd, nvfp4_moe_decode_fwd   out[t] = sum_j gate[t,j] W2[e] (silu(W1g[e] x_t) * (W1u[e] x_t))
//   mxfp8_matvec, nvfp4_matvec             y[t] = W x_t
//
// Mathematics.  Only the weights are low-precision; x (bf16) and the intermediate h (fp32) are not
// rounded to 8 or 4 bits.  Each activation is instead written as a short sum of numbers the
// tensor core takes beside those weights, and the terms become extra columns of one MMA:
//   MXFP8  the significand is cut into groups of 4 bits, each group an E4M3 number under its own
//          power-of-two block scale: x = x0 + x1 (8 significant bits: bf16 exactly), h = h0 + h1 + h2
//          (12 bits, the last group rounded to nearest).  Values below 2^-13 of their block's
//          largest lose bits below 2^-17 of it.
//   NVFP4  a block's values, scaled to |v| < 4, are written in base 8 with digits -4..4 (E2M1 holds
//          these integers): v = d0 + d1/8 + ... + d4/4096, an error of at most 2^-14 of the block's
//          largest value.
// Accumulation is fp32 in TMEM; the columns of one token are added in fp32 and the result is
// rounded once, to bf16.
//
// What bounds it: reading the weights once (a token's flops per weight byte are far below the tensor
// cores').  So the weights are the M operand: TMA brings 128 rows x 128 code bytes per K step and
// their scale atoms, the MMA reads both as stored, and no instruction is spent per weight.  The
// tokens are the N operand, converted by four warps while the weights travel.
//
// Split: one CTA takes a range of K steps of one 128-row tile; a cluster of up to 8 CTAs shares the
// tile and adds its partial sums through distributed shared memory in a fixed order (no atomics:
// results do not depend on timing).  Two CTAs share an SM so that one's start and end are hidden
// behind the other's copies.
//   k_decode<GATE_UP>  cluster = (gate, up) x K ranges of 128 columns of F of one active expert:
//                      h = gate silu(g) u, fp32 rows [token-expert pair, F]
//   k_decode<DOWN>     cluster = K ranges of 128 rows of H; K runs over all active experts' F one
//                      after the other with one column group per token (zero where the token did
//                      not choose the expert), so the accumulator itself sums a token's experts
//   k_decode<LINEAR>   cluster = K ranges of 128 rows of W
// DOWN is launched programmatically dependent on GATE_UP: its weight copies start while GATE_UP's
// last CTAs run; only its conversion warps wait for h.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cstdlib>

#include "mx_device.cuh"
#include "mx_internal.h"
#include "mxfp8moe.h"

namespace mx {
namespace {

constexpr int DEC_THREADS = 192;             // warp 0 copies, warp 1 MMA, warps 2-5 conversion + epilogue
constexpr int DEC_CONV_WARPS = 4;
constexpr int DEC_A_STAGE = 128 * 128;       // 128 weight rows x 128 code bytes
constexpr int DEC_MAX_TOKENS = 64;           // tokens of one call
constexpr int DEC_CHUNK = 32;                // most tokens of one accumulator (bits of an expert's token mask)
constexpr int DEC_MAX_K = 32;                // choices per token
constexpr int DEC_MAX_CLUSTER = 8;
constexpr int DEC_MAX_A = 8, DEC_MAX_B = 4;  // ring depths
// Two CTAs per SM: half of 228 KB each, less 1 KB the system keeps per CTA.
constexpr int DEC_SMEM = 113 * 1024;
constexpr uint32_t DEC_TMEM_COLS = 256;      // two CTAs per SM share 512
// TMEM columns: the accumulator (up to 160), then two sets of scales of A and of B, used in turn.
constexpr uint32_t DEC_SFA_COL = 160, DEC_SFB_COL = 192;
constexpr uint32_t DEC_BAR_CONV = 1;         // hardware barrier of the conversion warps

enum DecMode { DEC_GATE_UP = 0, DEC_DOWN = 1, DEC_LINEAR = 2 };
enum DecFmt { DEC_MX = 0, DEC_NV = 1 };

// Columns per token: E4M3 pieces of a bf16 (2) or fp32 (3) value, or base-8 digits (5).
constexpr int dec_pieces(int fmt, int mode) { return fmt == DEC_NV ? 5 : mode == DEC_DOWN ? 3 : 2; }
constexpr int dec_step_values(int fmt) { return fmt == DEC_NV ? 256 : 128; }
constexpr int dec_atoms(int fmt) { return fmt == DEC_NV ? 4 : 1; }   // scale atoms per 128 rows and step

// Shared memory of one CTA (byte offsets from a 1024-byte boundary).
struct DecLayout {
  int na, nb;                        // stages of the weight ring and of the activation ring
  int b_stage, sfb_stage;
  int b, sfa, sfb, bars, misc;       // the weight ring is at 0
};

struct DecParams {
  DecLayout L;
  const uint16_t* x;      // GATE_UP, LINEAR: bf16 [T, K]
  float* h;               // GATE_UP out, DOWN in: [T * k, F]
  float* hmax;            // NVFP4: largest |h| of every 32 columns, [T * k, F / 32]
  const uint8_t* w_sf;
  const float* w_amax;    // NVFP4
  const int32_t* experts; // [T, k]
  const float* gates;     // [T, k] or NULL
  uint16_t* out;          // DOWN: [T, H], LINEAR: [T, N]
  uint32_t* err;
  int T, k, E;
  int K;                  // contraction length of one weight row
  int steps;              // its K steps
  int kt;                 // its scale atoms per 128-row tile
  int tiles;              // 128-row tiles (of F, H or N)
  int F;
  int cs;                 // CTAs per cluster
  int per_chunk;          // tokens per chunk (blockIdx.y)
  uint64_t timeout_ns, drain_ns;
};

__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void conv_barrier() {
  asm volatile("bar.sync %0, %1;" ::"r"(DEC_BAR_CONV), "r"(DEC_CONV_WARPS * 32) : "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void tc_copy_sf(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}
__device__ __forceinline__ void tc_mma_nvf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
          d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// One thread waits; on a timeout it records the bit and raises the CTA's abort flag.
__device__ __forceinline__ bool dec_wait(uint64_t* bar, uint32_t parity, volatile int* abort, const DecParams& p,
                                         uint32_t err_bit) {
  if (mbar_wait_bounded(bar, parity, abort, p.timeout_ns)) return true;
  if (!*abort) atomicOr(p.err, err_bit);
  *abort = 1;
  return false;
}
__device__ __forceinline__ bool dec_warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, const DecParams& p,
                                              uint32_t err_bit, int lane) {
  int ok = 1;
  if (lane == 0) ok = dec_wait(bar, parity, abort, p, err_bit) ? 1 : 0;
  return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
}

// floor(log2) of a block's largest magnitude from its float bits, kept where the scales used below
// stay representable (blocks under 2^-100 are treated as if their largest value were 2^-100).
__device__ __forceinline__ int block_exponent(uint32_t abs_bits) {
  return max(static_cast<int>(abs_bits >> 23) - 127, -100);
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

template <int N>
__device__ __forceinline__ uint32_t abs_max_bits(const float (&v)[N]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

// Eight values of a 32-value block (four lanes hold the block) -> P E4M3 pieces: 8 code bytes in
// row p * tp + c of the step's activation tile and, from the block's first lane, the scale bytes.
// g: which eight of the step's 128 values.  Pieces 0..P-2 are cut (the residual is exact), the last
// is rounded to nearest even.
template <int P>
__device__ __forceinline__ void put_pieces_mx(const float (&v)[8], uint8_t* sB, uint8_t* sSF, int c, int tp, int g) {
  uint32_t m = abs_max_bits(v);
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  if (c < 0) return;
  const bool finite = m < 0x7F800000u;
  const int eb = block_exponent(m);
  const float inv = pow2f(7 - min(eb, 127));   // largest magnitude in [128, 256)
  const uint64_t inv2 = f2_pack(inv, inv), sixteen = f2_pack(16.0f, 16.0f), minus1 = f2_pack(-1.0f, -1.0f);
  uint64_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = f2_mul(f2_pack(v[2 * i], v[2 * i + 1]), inv2);
#pragma unroll
  for (int q = 0; q < P; ++q) {
    uint32_t code[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (q + 1 < P) {
        const uint64_t top = r[i] & 0xFFF00000FFF00000ull;   // sign, exponent, 3 bits after the leading one
        code[i] = e4m3x2_f2(top);
        r[i] = f2_mul(f2_fma(top, minus1, r[i]), sixteen);
      } else {
        code[i] = e4m3x2_f2(r[i]);
      }
    }
    const int row = q * tp + c;
    *reinterpret_cast<uint2*>(sB + row * 128 + (((g >> 1) ^ (row & 7)) << 4) + ((g & 1) << 3)) =
        make_uint2(code[0] | (code[1] << 16), code[2] | (code[3] << 16));
    if ((g & 3) == 0)   // 0xFF: NaN, the column of a token with a non-finite value
      sSF[(row >> 7) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (g >> 2)] =
          finite ? static_cast<uint8_t>(eb + 120 - 4 * q) : static_cast<uint8_t>(0xFF);
  }
}

// One 16-value block -> P base-8 digits as E2M1: 8 code bytes in row p * tp + c, and the block's UE4M3
// scale 2^(8 + e_block - e_token) (the same for every digit).  j: which of the step's 16 blocks.
template <int P>
__device__ __forceinline__ void put_pieces_nv(const float (&v)[16], int e_tok, uint8_t* sB, uint8_t* sSF, int nat,
                                              int c, int tp, int j) {
  const uint32_t m = abs_max_bits(v);
  const bool finite = m < 0x7F800000u;
  // blocks more than 2^17 below the token's largest value share the smallest scale
  const int eb = max(block_exponent(m), e_tok - 17);
  const float inv = pow2f(1 - min(eb, 127));   // largest magnitude in [2, 4)
  const uint64_t inv2 = f2_pack(inv, inv), eight = f2_pack(8.0f, 8.0f), minus8 = f2_pack(-8.0f, -8.0f);
  // adding and subtracting 1.5 * 2^23 rounds to the nearest integer
  const uint64_t big = f2_pack(12582912.0f, 12582912.0f), minus_big = f2_pack(-12582912.0f, -12582912.0f);
  uint64_t r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = f2_mul(f2_pack(v[2 * i], v[2 * i + 1]), inv2);
  const int d = eb - e_tok + 8;   // -9 .. 8
  const uint32_t sc = !finite ? 0x7Fu : d >= -6 ? static_cast<uint32_t>(d + 7) << 3 : 1u << (d + 9);
#pragma unroll
  for (int q = 0; q < P; ++q) {
    uint64_t n[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      n[i] = f2_add(f2_add(r[i], big), minus_big);
      if (q + 1 < P) r[i] = f2_fma(n[i], minus8, f2_mul(r[i], eight));
    }
    const int row = q * tp + c;
    uint2 w;
    w.x = e2m1x8(f2_lo(n[0]), f2_hi(n[0]), f2_lo(n[1]), f2_hi(n[1]), f2_lo(n[2]), f2_hi(n[2]), f2_lo(n[3]), f2_hi(n[3]));
    w.y = e2m1x8(f2_lo(n[4]), f2_hi(n[4]), f2_lo(n[5]), f2_hi(n[5]), f2_lo(n[6]), f2_hi(n[6]), f2_lo(n[7]), f2_hi(n[7]));
    *reinterpret_cast<uint2*>(sB + row * 128 + (((j >> 1) ^ (row & 7)) << 4) + ((j & 1) << 3)) = w;
    sSF[((j >> 2) * nat + (row >> 7)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (j & 3)] =
        static_cast<uint8_t>(sc);
  }
}

__device__ __forceinline__ void unpack8(const uint4 w, float* v) {
  v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
  v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
}

template <int FMT, int MODE>
__global__ void __launch_bounds__(DEC_THREADS, 2) k_decode(const __grid_constant__ CUtensorMap tm, const DecParams p) {
  constexpr int P = dec_pieces(FMT, MODE);
  constexpr int KSTEP = dec_step_values(FMT);
  constexpr int ATOMS = dec_atoms(FMT);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const DecLayout& L = p.L;
  uint64_t* full_a = reinterpret_cast<uint64_t*>(smem + L.bars);
  uint64_t* empty_a = full_a + DEC_MAX_A;
  uint64_t* full_b = empty_a + DEC_MAX_A;
  uint64_t* empty_b = full_b + DEC_MAX_B;
  uint64_t* done = empty_b + DEC_MAX_B;
  uint64_t* drained = done + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* s_nact = reinterpret_cast<int*>(tmem_holder + 2);
  int* s_tok = reinterpret_cast<int*>(smem + L.misc);            // GATE_UP: token of each column
  float* s_gate = reinterpret_cast<float*>(s_tok + DEC_CHUNK);   // GATE_UP: its routing weight
  int* s_emax = reinterpret_cast<int*>(s_gate + DEC_CHUNK);      // NVFP4: exponent of each column's scale
  uint32_t* s_mask = reinterpret_cast<uint32_t*>(s_emax + DEC_CHUNK);   // [E] tokens that chose the expert
  int* s_act_e = reinterpret_cast<int*>(s_mask + p.E);           // active experts: id, tokens, first row of h
  const int nact_max = min(p.E, p.per_chunk * p.k);
  uint32_t* s_act_m = reinterpret_cast<uint32_t*>(s_act_e + nact_max);
  int* s_act_off = reinterpret_cast<int*>(s_act_m + nact_max);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_cta_rank());
  const int cluster = blockIdx.x / p.cs;
  const int t0 = blockIdx.y * p.per_chunk;
  const int tc = min(p.per_chunk, p.T - t0);
  const bool first_cta = blockIdx.x == 0 && blockIdx.y == 0;

  // The error word starts at 0 here; a wait can run out only after the work below, in any CTA.
  if (MODE != DEC_DOWN && first_cta && tid == 0) *p.err = 0;
  if constexpr (MODE == DEC_GATE_UP) pdl_launch_dependents();
  if (tid == 0) {
    for (int s = 0; s < DEC_MAX_A; ++s) {
      mbar_init(&full_a[s], 1);
      mbar_init(&empty_a[s], 1);
    }
    for (int s = 0; s < DEC_MAX_B; ++s) {
      mbar_init(&full_b[s], DEC_CONV_WARPS / L.nb);
      mbar_init(&empty_b[s], 1);
    }
    mbar_init(done, 1);
    mbar_init(drained, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, DEC_TMEM_COLS);
    tmem_relinquish();
  }
  if (warp >= 2) {   // unused columns hold zero codes, never stale bytes
    for (int i = tid - 64; i < (L.nb * (L.b_stage + L.sfb_stage)) / 16; i += DEC_CONV_WARPS * 32) {
      const int off = i * 16;
      *reinterpret_cast<uint4*>(off < L.nb * L.b_stage ? smem + L.b + off : smem + L.sfb + (off - L.nb * L.b_stage)) =
          make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
  }

  // ---- routing: which tokens of the chunk chose which expert, and the list of chosen experts ----
  int nact = 1;
  if constexpr (MODE != DEC_LINEAR) {
    for (int e = tid; e < p.E; e += DEC_THREADS) s_mask[e] = 0;
    __syncthreads();
    for (int i = tid; i < tc * p.k; i += DEC_THREADS) {
      const int e = __ldg(p.experts + static_cast<int64_t>(t0) * p.k + i);
      if (e >= 0 && e < p.E) atomicOr(&s_mask[e], 1u << (i / p.k));
    }
    if (MODE == DEC_GATE_UP && first_cta)
      for (int i = tid; i < p.T * p.k; i += DEC_THREADS)
        if (__ldg(p.experts + i) >= p.E) atomicOr(p.err, ERR_EXPERT_RANGE);
    __syncthreads();
    if (warp == 0) {
      int n = 0, rows = t0 * p.k;
      for (int base = 0; base < p.E; base += 32) {
        const uint32_t m = base + lane < p.E ? s_mask[base + lane] : 0u;
        const uint32_t act = __ballot_sync(0xFFFFFFFFu, m != 0);
        int incl = __popc(m);
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
          if (lane >= d) incl += o;
        }
        if (m != 0) {
          const int pos = n + __popc(act & ((1u << lane) - 1u));
          s_act_e[pos] = base + lane;
          s_act_m[pos] = m;
          s_act_off[pos] = rows + incl - __popc(m);
        }
        n += __popc(act);
        rows += __shfl_sync(0xFFFFFFFFu, incl, 31);
      }
      if (lane == 0) *s_nact = n;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  if constexpr (MODE != DEC_LINEAR) nact = *s_nact;

  // ---- this CTA's tile and K range ----
  int a0 = 0, tile = cluster;
  if constexpr (MODE == DEC_GATE_UP) {
    a0 = cluster / p.tiles;
    tile = cluster - a0 * p.tiles;
    if (a0 >= nact) {   // fewer experts were chosen than could be: the whole cluster leaves
      if (warp == 1) tmem_dealloc(tmem, DEC_TMEM_COLS);
      return;
    }
  }
  int ncol = tc;          // token columns
  uint32_t mask0 = 0;
  if constexpr (MODE == DEC_GATE_UP) {
    mask0 = s_act_m[a0];
    ncol = __popc(mask0);
  }
  const int tp = (ncol + 7) & ~7;
  const int n_mma = (P * tp + 15) & ~15;
  const int nat = (n_mma + 127) >> 7;    // scale atoms of B per MMA
  const int ns = MODE == DEC_GATE_UP ? p.cs >> 1 : p.cs;
  const int si = MODE == DEC_GATE_UP ? rank >> 1 : rank;
  const int total = MODE == DEC_DOWN ? nact * p.steps : p.steps;
  const int s_begin = static_cast<int>(static_cast<int64_t>(total) * si / ns);
  const int n_steps = static_cast<int>(static_cast<int64_t>(total) * (si + 1) / ns) - s_begin;

  if (warp == 0) {
    // ---------------- weight copies (lane 0) ----------------
    if (lane == 0) {
      int a = MODE == DEC_DOWN && p.steps > 0 ? s_begin / p.steps : a0;
      int f = s_begin - (MODE == DEC_DOWN ? a * p.steps : 0);
      int issued = 0;
      for (int i = 0; i < n_steps; ++i) {
        const int slot = i % L.na;
        if (i >= L.na && !dec_wait(&empty_a[slot], ((i / L.na) - 1) & 1, abort_flag, p, ERR_TIMEOUT_PRODUCER)) break;
        int64_t row = static_cast<int64_t>(tile) * 128;
        if constexpr (MODE == DEC_GATE_UP)
          row += static_cast<int64_t>(s_act_e[a]) * 2 * p.F + static_cast<int64_t>(rank & 1) * p.F;
        if constexpr (MODE == DEC_DOWN) row += static_cast<int64_t>(s_act_e[a]) * p.tiles * 128;
        mbar_arrive_expect_tx(&full_a[slot], DEC_A_STAGE + ATOMS * 512);
        tma_load_2d(smem + slot * DEC_A_STAGE, &tm, &full_a[slot], f * 128, static_cast<int32_t>(row));
        bulk_load(smem + L.sfa + slot * ATOMS * 512,
                  p.w_sf + ((row >> 7) * p.kt + static_cast<int64_t>(f) * ATOMS) * 512, ATOMS * 512, &full_a[slot]);
        ++issued;
        if (++f == p.steps) {
          f = 0;
          ++a;
        }
      }
      // every copy must have landed before the CTA may exit or its stages are reused
      for (int i = max(0, issued - L.na); i < issued; ++i)
        if (!mbar_wait_bounded(&full_a[i % L.na], (i / L.na) & 1, nullptr, p.drain_ns))
          atomicOr(p.err, ERR_TIMEOUT_DRAIN);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- scale copies and MMAs (lane 0) ----------------
    if (lane == 0) {
      const uint32_t idesc = FMT == DEC_NV ? idesc_nvf4(128, n_mma) : idesc_mxf8_e4m3(128, n_mma);
      bool ok = true, any = false;
      for (int i = 0; i < n_steps; ++i) {
        const int slot = i % L.na, bs = i % L.nb;
        if (!dec_wait(&full_a[slot], (i / L.na) & 1, abort_flag, p, ERR_TIMEOUT_MMA) ||
            !dec_wait(&full_b[bs], (i / L.nb) & 1, abort_flag, p, ERR_TIMEOUT_MMA) ||
            // the scale columns about to be overwritten were last read by step i - 2's MMAs
            (i >= 2 && !dec_wait(&empty_a[(i - 2) % L.na], ((i - 2) / L.na) & 1, abort_flag, p, ERR_TIMEOUT_MMA))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sa = smem_u32(smem + slot * DEC_A_STAGE), sb = smem_u32(smem + L.b + bs * L.b_stage);
        const uint32_t sfa = smem_u32(smem + L.sfa + slot * ATOMS * 512);
        const uint32_t sfb = smem_u32(smem + L.sfb + bs * L.sfb_stage);
        const uint32_t t_sfa = tmem + DEC_SFA_COL + (i & 1) * 16, t_sfb = tmem + DEC_SFB_COL + (i & 1) * 32;
#pragma unroll
        for (int m = 0; m < ATOMS; ++m) {
          tc_copy_sf(t_sfa + 4 * m, sdesc_sf_atom(sfa + 512 * m));
          for (int j = 0; j < nat; ++j)
            tc_copy_sf(t_sfb + 8 * m + 4 * j, sdesc_sf_atom(sfb + 512 * (m * nat + j)));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (FMT == DEC_NV)
            tc_mma_nvf4(tmem, sdesc_kmajor_sw128(sa + 32 * k), sdesc_kmajor_sw128(sb + 32 * k), idesc, t_sfa + 4 * k,
                        t_sfb + 8 * k, (i | k) != 0 ? 1u : 0u);
          else
            tc_mma_mxf8(tmem, sdesc_kmajor_sw128(sa + 32 * k), sdesc_kmajor_sw128(sb + 32 * k),
                        idesc_with_sf_id(idesc, k), t_sfa, t_sfb, (i | k) != 0 ? 1u : 0u);
        }
        tc_commit(&empty_a[slot]);
        tc_commit(&empty_b[bs]);
        any = true;
      }
      if (ok && any) tc_commit(done);
      else if (ok) mbar_arrive(done);
      if (any) {
        tc_commit(drained);
        if (!mbar_wait_bounded(drained, 0, nullptr, p.drain_ns)) atomicOr(p.err, ERR_TIMEOUT_DRAIN);
      }
    }
    __syncwarp();
  } else {
    // ---------------- activations -> columns of the MMA ----------------
    const int cw = warp - 2, ct = tid - 64;
    if constexpr (MODE == DEC_DOWN) pdl_wait();   // h is GATE_UP's
    if constexpr (MODE == DEC_GATE_UP) {
      if (ct < ncol) {
        uint32_t m = mask0;
        for (int i = 0; i < ct; ++i) m &= m - 1u;
        const int t = __ffs(m) - 1;
        s_tok[ct] = t;
        // a token that lists the expert more than once: the weights add
        float w = 0.0f;
        for (int j = 0; j < p.k; ++j) {
          const int64_t q = static_cast<int64_t>(t0 + t) * p.k + j;
          if (__ldg(p.experts + q) == s_act_e[a0]) w += p.gates != nullptr ? __ldg(p.gates + q) : 1.0f;
        }
        s_gate[ct] = w;
      }
      conv_barrier();
    }
    // row of x (or of h, -1 where the token did not choose expert a) behind column c
    auto src_row = [&](int c, int a) -> int64_t {
      if constexpr (MODE == DEC_GATE_UP) return t0 + s_tok[c];
      if constexpr (MODE == DEC_LINEAR) return t0 + c;
      const uint32_t m = s_act_m[a];
      return (m >> c) & 1u ? s_act_off[a] + __popc(m & ((1u << c) - 1u)) : -1;
    };
    if constexpr (FMT == DEC_NV) {
      // exponent of each column's largest magnitude over this CTA's K range: one scale per column
      // and CTA (the ranges' partial sums are added after scaling)
      for (int c = cw; c < ncol; c += DEC_CONV_WARPS) {
        uint32_t m = 0;
        if constexpr (MODE == DEC_DOWN) {
          const int tiles32 = p.F / 32;
          for (int s = s_begin; s < s_begin + n_steps;) {
            const int a = s / p.steps, f = s - a * p.steps;
            const int nf = min(p.steps - f, s_begin + n_steps - s);
            const int64_t r = src_row(c, a);
            if (r >= 0)
              for (int i = f * 8 + lane; i < min((f + nf) * 8, tiles32); i += 32)
                m = max(m, __float_as_uint(p.hmax[r * tiles32 + i]));
            s += nf;
          }
        } else {
          const uint16_t* xr = p.x + src_row(c, 0) * p.K;
          const int k1 = min((s_begin + n_steps) * KSTEP, p.K);
          for (int k = s_begin * KSTEP + lane * 8; k < k1; k += 256) {
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(xr + k));
            const uint32_t q = __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                        __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
            m = max(m, max(q & 0xFFFFu, q >> 16) << 16);
          }
        }
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if (lane == 0) s_emax[c] = block_exponent(m);
      }
    }
    if constexpr (FMT == DEC_NV) conv_barrier();   // s_emax

    const int group = cw % L.nb, sub = cw / L.nb, nsub = DEC_CONV_WARPS / L.nb;   // ring slot = group
    const int g = lane & 15;
    for (int i = group; i < n_steps; i += L.nb) {
      if (i >= L.nb &&
          !dec_warp_wait(&empty_b[group], ((i / L.nb) - 1) & 1, abort_flag, p, ERR_TIMEOUT_SF, lane))
        break;
      uint8_t* sB = smem + L.b + group * L.b_stage;
      uint8_t* sSF = smem + L.sfb + group * L.sfb_stage;
      const int s = s_begin + i;
      const int a = MODE == DEC_DOWN ? s / p.steps : a0;
      const int f = MODE == DEC_DOWN ? s - a * p.steps : s;
      for (int c0 = 2 * sub; c0 < ncol; c0 += 2 * nsub) {
        const int c = c0 + (lane >> 4);
        const int64_t r = c < ncol ? src_row(c, a) : -1;
        if constexpr (FMT == DEC_MX) {
          float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
          if (r >= 0) {
            const int64_t o = r * p.K + f * KSTEP + g * 8;
            if constexpr (MODE == DEC_DOWN) {
              const float4 u0 = *reinterpret_cast<const float4*>(p.h + o);
              const float4 u1 = *reinterpret_cast<const float4*>(p.h + o + 4);
              v[0] = u0.x; v[1] = u0.y; v[2] = u0.z; v[3] = u0.w;
              v[4] = u1.x; v[5] = u1.y; v[6] = u1.z; v[7] = u1.w;
            } else {
              unpack8(__ldg(reinterpret_cast<const uint4*>(p.x + o)), v);
            }
          }
          put_pieces_mx<P>(v, sB, sSF, c < ncol ? c : -1, tp, g);
        } else {
          float v[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) v[q] = 0.0f;
          const int kk = f * KSTEP + g * 16;
          if (r >= 0 && kk < p.K) {
            const int64_t o = r * p.K + kk;
            if constexpr (MODE == DEC_DOWN) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const float4 u = *reinterpret_cast<const float4*>(p.h + o + 4 * q);
                v[4 * q] = u.x; v[4 * q + 1] = u.y; v[4 * q + 2] = u.z; v[4 * q + 3] = u.w;
              }
            } else {
              unpack8(__ldg(reinterpret_cast<const uint4*>(p.x + o)), v);
              unpack8(__ldg(reinterpret_cast<const uint4*>(p.x + o + 8)), v + 8);
            }
          }
          if (c < ncol) put_pieces_nv<P>(v, s_emax[c], sB, sSF, nat, c, tp, g);
        }
      }
      fence_proxy_async_smem();   // the tensor core reads these bytes through the async proxy
      __syncwarp();
      if (lane == 0) mbar_arrive(&full_b[group]);
    }

    // ---------------- accumulator -> this CTA's partial sums [column][128 rows] ----------------
    if (dec_warp_wait(done, 0, abort_flag, p, ERR_TIMEOUT_EPILOGUE, lane)) {
      tc_fence_after();
      const int quarter = warp & 3, row = quarter * 32 + lane;
      const uint32_t t_row = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
      float* part = reinterpret_cast<float*>(smem);   // the weight ring: all its copies have been consumed
      float alpha = 1.0f;
      if constexpr (FMT == DEC_NV) alpha = 1.0f / nv_encode_scale(__ldg(p.w_amax));
      for (int c0 = 0; c0 < ncol; c0 += 8) {
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (n_steps > 0) {
          uint32_t d[P][8];
#pragma unroll
          for (int q = 0; q < P; ++q) tmem_ld_32x32b_x8(t_row + q * tp + c0, d[q]);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            v[j] = __uint_as_float(d[P - 1][j]);
#pragma unroll
            for (int q = P - 2; q >= 0; --q)   // smallest first; a digit's place is 1/8 of the one before
              v[j] = FMT == DEC_NV ? fmaf(v[j], 0.125f, __uint_as_float(d[q][j])) : v[j] + __uint_as_float(d[q][j]);
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c0 + j < ncol)
            part[(c0 + j) * 128 + row] =
                FMT == DEC_NV ? ldexpf(v[j] * alpha, s_emax[c0 + j] - 9) : v[j];
      }
    }
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync_all();

  // ---------------- sum over the cluster's K ranges, finish columns rank, rank + cs, ... ----------------
  if (warp >= 2) {
    const int row = (warp & 3) * 32 + lane;
    const float* part = reinterpret_cast<const float*>(smem);
    for (int c = rank; c < ncol; c += p.cs) {
      const float* mine = part + c * 128 + row;
      if constexpr (MODE == DEC_GATE_UP) {
        float gs = 0.0f, us = 0.0f;
        for (int q = 0; q < ns; ++q) {
          gs += ld_cluster_f32(map_to_cta(mine, 2 * q));
          us += ld_cluster_f32(map_to_cta(mine, 2 * q + 1));
        }
        const float hv = s_gate[c] * (gs / (1.0f + expf(-gs))) * us;
        const int64_t hr = s_act_off[a0] + c;
        p.h[hr * p.F + tile * 128 + row] = hv;
        if constexpr (FMT == DEC_NV) {
          const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(hv) & 0x7FFFFFFFu);
          if (lane == 0) p.hmax[hr * (p.F / 32) + tile * 4 + (warp & 3)] = __uint_as_float(m);
        }
      } else {
        float v = 0.0f;
        for (int q = 0; q < ns; ++q) v += ld_cluster_f32(map_to_cta(mine, q));
        p.out[static_cast<int64_t>(t0 + c) * p.tiles * 128 + tile * 128 + row] =
            static_cast<uint16_t>(pack_bf16x2(v, 0.0f) & 0xFFFFu);
      }
    }
  }
  __syncwarp();
  cluster_sync_all();   // no CTA leaves while another reads its partial sums
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, DEC_TMEM_COLS);
  }
}

// ---- host side -------------------------------------------------------------------------------

constexpr uint64_t kDecWaitNs = 2000000000ull;   // 2 s per wait; teardown waits always keep it

// Limit of every pipeline wait: kDecWaitNs, or MXFP8MOE_WAIT_LIMIT_NS as for the grouped GEMMs.
uint64_t dec_wait_ns() {
  const char* v = getenv("MXFP8MOE_WAIT_LIMIT_NS");
  if (v == nullptr || *v == 0) return kDecWaitNs;
  char* end = nullptr;
  const unsigned long long n = strtoull(v, &end, 10);
  return (end != nullptr && *end == 0 && n > 0) ? static_cast<uint64_t>(n) : kDecWaitNs;
}

// 2-D byte matrix [rows, cols] (row pitch = cols) in boxes of 128 rows x 128 bytes, 128-byte swizzle.
bool make_weight_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols) {
  static std::atomic<void*> entry{nullptr};
  void* fn = entry.load(std::memory_order_acquire);
  if (fn == nullptr) {
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || fn == nullptr)
      return false;
    entry.store(fn, std::memory_order_release);
  }
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {cols};
  const cuuint32_t box[2] = {128, 128}, estr[2] = {1, 1};
  return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn)(
             m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int round_up(int v, int m) { return (v + m - 1) / m * m; }

// Shared memory for chunks of `tokens` tokens; false when fewer than 3 weight stages fit.
bool dec_layout(int fmt, int mode, int tokens, int E, int nact, DecLayout* out) {
  const int n = round_up(dec_pieces(fmt, mode) * round_up(tokens, 8), 16);
  DecLayout L{};
  L.b_stage = n * 128;
  L.sfb_stage = dec_atoms(fmt) * ((n + 127) / 128) * 512;
  // four activation stages (one per conversion warp) unless they would take the weights' room
  L.nb = 4 * (L.b_stage + L.sfb_stage) <= 40 * 1024 ? 4 : 2;
  const int misc = 3 * DEC_CHUNK * 4 + (mode == DEC_LINEAR ? 0 : E * 4 + nact * 12);
  const int fixed = L.nb * (L.b_stage + L.sfb_stage) + 256 + round_up(misc, 16);
  const int sfa = dec_atoms(fmt) * 512;
  L.na = std::min(DEC_MAX_A, (DEC_SMEM - 1024 - fixed) / (DEC_A_STAGE + sfa));
  if (L.na < 3) return false;
  L.b = L.na * DEC_A_STAGE;
  L.sfb = L.b + L.nb * L.b_stage;
  L.sfa = L.sfb + L.nb * L.sfb_stage;
  L.bars = L.sfa + L.na * sfa;
  L.misc = L.bars + 256;
  *out = L;
  return true;
}

// Per-device set-up of one kernel instance: dynamic shared memory, and the carve-out that lets two
// CTAs share an SM.
template <int FMT, int MODE>
bool dec_setup() {
  constexpr int kMaxDevices = 64;
  static std::atomic<bool> done[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
  if (done[dev]) return true;
  if (cudaFuncSetAttribute(k_decode<FMT, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, DEC_SMEM) != cudaSuccess ||
      cudaFuncSetAttribute(k_decode<FMT, MODE>, cudaFuncAttributePreferredSharedMemoryCarveout,
                           cudaSharedmemCarveoutMaxShared) != cudaSuccess)
    return false;
  done[dev] = true;
  return true;
}

template <int FMT, int MODE>
bool dec_launch(const CUtensorMap& tm, const DecParams& p, int clusters, int chunks, bool dependent,
                cudaStream_t stream) {
  if (!dec_setup<FMT, MODE>()) return false;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters) * p.cs, static_cast<unsigned>(chunks), 1);
  cfg.blockDim = dim3(DEC_THREADS, 1, 1);
  cfg.dynamicSmemBytes = DEC_SMEM;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_decode<FMT, MODE>, tm, p) == cudaSuccess;
}

// CTAs that share one 128-row tile's K steps: as many (1, 2, 4, 8) as keep at least `min_steps` steps
// each while the grid has fewer than two CTAs per SM on average.
int dec_split(int64_t tiles, int64_t steps, int max_split, int min_steps) {
  int ns = 1;
  while (2 * ns <= max_split && tiles * ns < 2 * 304 && steps >= static_cast<int64_t>(2 * ns) * min_steps) ns *= 2;
  return ns;
}

// Chunks of equal size (at most DEC_CHUNK tokens, fewer where their shared memory does not fit).
bool dec_chunks(int fmt, int mode, int T, int k, int E, DecLayout* L, int* per_chunk, int* chunks) {
  for (int cap = DEC_CHUNK; cap >= 8; cap -= 8) {
    *chunks = (T + cap - 1) / cap;
    *per_chunk = (T + *chunks - 1) / *chunks;
    if (dec_layout(fmt, mode, *per_chunk, E, std::min(E, *per_chunk * k), L)) return true;
  }
  return false;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
constexpr size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

struct DecWs {
  size_t h, hmax, total;
};
bool dec_ws_layout(int64_t T, int k, int64_t H, int64_t F, int E, DecWs* out) {
  if (T < 0 || T > DEC_MAX_TOKENS || k < 1 || k > DEC_MAX_K || E < 1 || E > 1024 || H <= 0 || F <= 0 || F > INT32_MAX)
    return false;
  DecWs w{};
  w.h = 256;
  w.hmax = align256(w.h + static_cast<size_t>(T) * k * F * sizeof(float));
  w.total = align256(w.hmax + static_cast<size_t>(T) * k * ((F + 31) / 32) * sizeof(float));
  *out = w;
  return true;
}

template <int FMT>
int moe_decode(const void* x, int64_t T, int64_t H, int64_t F, int E, int k, const int32_t* experts,
               const float* gates, const uint8_t* w1_q, const uint8_t* w1_sf, const float* w1_amax,
               const uint8_t* w2_q, const uint8_t* w2_sf, const float* w2_amax, void* out, void* workspace,
               size_t workspace_bytes, void* stream) {
  if (T < 0 || E < 1 || E > 1024 || k < 1 || H <= 0 || F <= 0) return MXFP8_ERR_INVALID_ARG;
  if (T > DEC_MAX_TOKENS || k > DEC_MAX_K || H % 128 != 0 || F % 128 != 0) return MXFP8_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(E) * 2 * F > INT32_MAX || static_cast<int64_t>(E) * H > INT32_MAX)
    return MXFP8_ERR_UNSUPPORTED;
  DecWs ws;
  if (!dec_ws_layout(T, k, H, F, E, &ws)) return MXFP8_ERR_UNSUPPORTED;
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < ws.total)
    return workspace == nullptr ? MXFP8_ERR_INVALID_ARG : MXFP8_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0)
    return cudaMemsetAsync(workspace, 0, sizeof(uint32_t), s) == cudaSuccess ? MXFP8_OK : MXFP8_ERR_CUDA;
  const void* ptrs[] = {x, w1_q, w1_sf, w2_q, w2_sf, out};
  for (const void* q : ptrs)
    if (q == nullptr || !aligned16(q)) return MXFP8_ERR_INVALID_ARG;
  if (experts == nullptr || (reinterpret_cast<uintptr_t>(experts) & 3u) != 0 ||
      (reinterpret_cast<uintptr_t>(gates) & 3u) != 0)
    return MXFP8_ERR_INVALID_ARG;
  if (FMT == DEC_NV && (w1_amax == nullptr || w2_amax == nullptr)) return MXFP8_ERR_INVALID_ARG;

  const int bytes_per_2 = FMT == DEC_NV ? 1 : 2;   // code bytes of two values
  CUtensorMap m1, m2;
  if (!make_weight_map(&m1, w1_q, static_cast<uint64_t>(E) * 2 * F, static_cast<uint64_t>(H) * bytes_per_2 / 2) ||
      !make_weight_map(&m2, w2_q, static_cast<uint64_t>(E) * H, static_cast<uint64_t>(F) * bytes_per_2 / 2))
    return MXFP8_ERR_CUDA;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  const int ks = dec_step_values(FMT);
  DecParams p{};
  p.x = static_cast<const uint16_t*>(x);
  p.h = reinterpret_cast<float*>(w + ws.h);
  p.hmax = reinterpret_cast<float*>(w + ws.hmax);
  p.experts = experts;
  p.gates = gates;
  p.out = static_cast<uint16_t*>(out);
  p.err = reinterpret_cast<uint32_t*>(w);
  p.T = static_cast<int>(T);
  p.k = k;
  p.E = E;
  p.F = static_cast<int>(F);
  p.timeout_ns = dec_wait_ns();
  p.drain_ns = kDecWaitNs;
  int chunks = 0;
  // one chunking for both kernels: DOWN (more columns per token) has the tighter layout
  if (!dec_chunks(FMT, DEC_DOWN, p.T, k, E, &p.L, &p.per_chunk, &chunks)) return MXFP8_ERR_UNSUPPORTED;
  const DecLayout down = p.L;
  const int nact = std::min(E, p.per_chunk * k);
  if (!dec_layout(FMT, DEC_GATE_UP, p.per_chunk, E, nact, &p.L)) return MXFP8_ERR_UNSUPPORTED;

  p.w_sf = w1_sf;
  p.w_amax = w1_amax;
  p.K = static_cast<int>(H);
  p.steps = static_cast<int>((H + ks - 1) / ks);
  p.kt = p.steps * dec_atoms(FMT);
  p.tiles = static_cast<int>(F / 128);
  const int64_t clusters = static_cast<int64_t>(nact) * p.tiles;
  p.cs = 2 * dec_split(2 * clusters * chunks, p.steps, DEC_MAX_CLUSTER / 2, 2);
  if (clusters * p.cs > INT32_MAX) return MXFP8_ERR_UNSUPPORTED;
  if (!dec_launch<FMT, DEC_GATE_UP>(m1, p, static_cast<int>(clusters), chunks, false, s)) return MXFP8_ERR_CUDA;

  p.L = down;
  p.w_sf = w2_sf;
  p.w_amax = w2_amax;
  p.K = static_cast<int>(F);
  p.steps = static_cast<int>((F + ks - 1) / ks);
  p.kt = p.steps * dec_atoms(FMT);
  p.tiles = static_cast<int>(H / 128);
  p.cs = dec_split(static_cast<int64_t>(p.tiles) * chunks, static_cast<int64_t>(nact) * p.steps, DEC_MAX_CLUSTER, 2);
  if (!dec_launch<FMT, DEC_DOWN>(m2, p, p.tiles, chunks, true, s)) return MXFP8_ERR_CUDA;
  return MXFP8_OK;
}

template <int FMT>
int matvec(const void* x, int64_t T, int64_t K, int64_t N, const uint8_t* w_q, const uint8_t* w_sf,
           const float* w_amax, void* y, void* workspace, size_t workspace_bytes, void* stream) {
  if (T < 0 || K <= 0 || N < 0) return MXFP8_ERR_INVALID_ARG;
  if (T > DEC_MAX_TOKENS || K % 128 != 0 || N % 128 != 0 || K > INT32_MAX || N > INT32_MAX)
    return MXFP8_ERR_UNSUPPORTED;
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0) return MXFP8_ERR_INVALID_ARG;
  if (workspace_bytes < matvec_workspace_size()) return MXFP8_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0 || N == 0)
    return cudaMemsetAsync(workspace, 0, sizeof(uint32_t), s) == cudaSuccess ? MXFP8_OK : MXFP8_ERR_CUDA;
  const void* ptrs[] = {x, w_q, w_sf, y};
  for (const void* q : ptrs)
    if (q == nullptr || !aligned16(q)) return MXFP8_ERR_INVALID_ARG;
  if (FMT == DEC_NV && w_amax == nullptr) return MXFP8_ERR_INVALID_ARG;
  CUtensorMap m;
  if (!make_weight_map(&m, w_q, static_cast<uint64_t>(N), static_cast<uint64_t>(K) / (FMT == DEC_NV ? 2 : 1)))
    return MXFP8_ERR_CUDA;
  const int ks = dec_step_values(FMT);
  DecParams p{};
  p.x = static_cast<const uint16_t*>(x);
  p.w_sf = w_sf;
  p.w_amax = w_amax;
  p.out = static_cast<uint16_t*>(y);
  p.err = static_cast<uint32_t*>(workspace);
  p.T = static_cast<int>(T);
  p.k = 1;
  p.K = static_cast<int>(K);
  p.steps = static_cast<int>((K + ks - 1) / ks);
  p.kt = p.steps * dec_atoms(FMT);
  p.tiles = static_cast<int>(N / 128);
  p.timeout_ns = dec_wait_ns();
  p.drain_ns = kDecWaitNs;
  int chunks = 0;
  if (!dec_chunks(FMT, DEC_LINEAR, p.T, 1, 0, &p.L, &p.per_chunk, &chunks)) return MXFP8_ERR_UNSUPPORTED;
  p.cs = dec_split(static_cast<int64_t>(p.tiles) * chunks, p.steps, DEC_MAX_CLUSTER, 2);
  return dec_launch<FMT, DEC_LINEAR>(m, p, p.tiles, chunks, false, s) ? MXFP8_OK : MXFP8_ERR_CUDA;
}

}  // namespace
}  // namespace mx

using namespace mx;

extern "C" {

size_t moe_decode_workspace_size(int64_t T, int k, int64_t H, int64_t F, int E) {
  DecWs w;
  return dec_ws_layout(T, k, H, F, E, &w) ? w.total : 0;
}

int moe_decode_fwd(const void* x, int64_t T, int64_t H, int64_t F, int E, int k, const int32_t* experts,
                   const float* gates, const uint8_t* w1_q, const uint8_t* w1_sf, const uint8_t* w2_q,
                   const uint8_t* w2_sf, void* out, void* workspace, size_t workspace_bytes, void* stream) {
  return moe_decode<DEC_MX>(x, T, H, F, E, k, experts, gates, w1_q, w1_sf, nullptr, w2_q, w2_sf, nullptr, out,
                            workspace, workspace_bytes, stream);
}

int nvfp4_moe_decode_fwd(const void* x, int64_t T, int64_t H, int64_t F, int E, int k, const int32_t* experts,
                         const float* gates, const uint8_t* w1_q, const uint8_t* w1_sf, const float* w1_amax,
                         const uint8_t* w2_q, const uint8_t* w2_sf, const float* w2_amax, void* out, void* workspace,
                         size_t workspace_bytes, void* stream) {
  return moe_decode<DEC_NV>(x, T, H, F, E, k, experts, gates, w1_q, w1_sf, w1_amax, w2_q, w2_sf, w2_amax, out,
                            workspace, workspace_bytes, stream);
}

size_t matvec_workspace_size(void) { return 256; }

int mxfp8_matvec(const void* x, int64_t T, int64_t K, int64_t N, const uint8_t* w_q, const uint8_t* w_sf, void* y,
                 void* workspace, size_t workspace_bytes, void* stream) {
  return matvec<DEC_MX>(x, T, K, N, w_q, w_sf, nullptr, y, workspace, workspace_bytes, stream);
}

int nvfp4_matvec(const void* x, int64_t T, int64_t K, int64_t N, const uint8_t* w_q, const uint8_t* w_sf,
                 const float* w_amax, void* y, void* workspace, size_t workspace_bytes, void* stream) {
  return matvec<DEC_NV>(x, T, K, N, w_q, w_sf, w_amax, y, workspace, workspace_bytes, stream);
}

}  // extern "C"

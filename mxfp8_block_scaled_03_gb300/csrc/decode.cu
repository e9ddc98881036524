// decode.cu -- the expert MLP and plain linears for a few tokens (decode steps): a whole MoE layer and
// y = x W^T for a few rows of x, from the MXFP8 and NVFP4 weights the grouped GEMMs use (same codes, same
// tensor-core scale layout).
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
//          largest value.  Its scale is relative to the row's largest block and reaches 2^-17 of it; a smaller block
//          is written under that scale, in its lower digits, with an error of at most 2^-31 of the row's largest more.
// Accumulation is fp32 in TMEM; the columns of one token are added in fp32 and the result is
// rounded once, to bf16.
//
// What bounds it: reading the weights once (a token's flops per weight byte are far below the tensor
// cores').  So the weights are the M operand: TMA brings 128 rows x 128 code bytes per K step and
// their scale atoms, the MMA reads both as stored, and no instruction is spent per weight.  The
// tokens are the N operand.  A (token, expert) pair is a row of activations; pairs are numbered expert after
// expert, so that an expert's columns are one box of the copy.
//   k_split_x        x -> columns (by token, or by pair for the MoE layer), and the bookkeeping of the call
//   k_decode<UP>     units: 128 columns of F of one chosen expert (and up to 16 or 32 of its tokens); gate
//                    and up rows are alternate K steps on two accumulators; h = gate silu(g) u -> columns
//   k_lift_low_blocks  NVFP4: small blocks of h under the smallest scale
//   k_decode<DOWN>   units: 128 rows of H of one chosen expert; a row of partial results per pair
//   k_sum_rows       adds a token's pairs
//   k_decode<LINEAR> units: 128 rows of W
// The kernels are launched programmatically dependent: a kernel's weight copies start while the one
// before it runs, and only what reads its results waits.  Weights are copied evict-first, so that everything
// else stays in L2 (NVFP4, 64 experts 2048x1408, 64 tokens: 69 us, 75 without).
// Two CTAs share an SM.  A CTA is bound by its own instructions, 0.2-0.4 us a K step of 16 KB (the MMA thread,
// and the warps that turn exponents into scales), an SM draws a step from memory in 0.35 us, and a kernel's
// first and last microseconds have one CTA's latencies.  One CTA per SM with twice the stages: 200 us against 158
// (MoE, NVFP4, 8 experts 4096x14336, 64 tokens), 28.2 against 26.5 (linear, MXFP8, 61x4096->28672), within 6%
// for 1 to 16 tokens (dec_layout says where it is used all the same).
// Measured (replayed graph, every call on other weights; share of the 6.77 TB/s a copy reaches):
//   MoE 8 experts 4096x14336, k 2    MXFP8  1 token 67.1 us (80%), 16 224 (96%), 64 229 (94%)
//                                    NVFP4  1 token 42.5 us (69%), 16 130 (90%), 64 144 to 159 (74 to 82%: by how the
//                                           tokens fall into groups of 16)
//   MoE 64 experts 2048x1408, k 8    MXFP8  1 token 24.1 us (44%), 8 67.1 (84%), 64 101.6 (83%)
//                                    NVFP4  1 token 20.7 us (28%), 8 45.7 (67%), 64 69.9 (66%)
//   linear 4096->28672               MXFP8  1 token 22.7 us (79%), 61 27.3 (68%)
//                                    NVFP4  1 token 14.7 us (67%), 61 21.5 (48%)
//   linear 1x4096->4096              MXFP8  8.5 us, NVFP4 7.5: launch, columns, first weights, parts, in a row
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cstdlib>

#include "launch_host.h"
#include "mx_device.cuh"
#include "mx_internal.h"
#include "mxfp8moe.h"

namespace mx {
namespace {

constexpr int DEC_A_STAGE = 128 * 128;       // 128 weight rows x 128 code bytes
constexpr int DEC_MAX_TOKENS = 64;           // tokens of one call
constexpr int DEC_MAX_K = 32;                // choices per token
constexpr int DEC_MAX_STAGES = 12;
// K values that make a CTA worth having in a shared unit: 4 steps of NVFP4, 8 of MXFP8.  Half as many cost 0.7 us
// (1x4096->4096) and 1.4 us (one token on 64 experts 2048x1408) more in either format, twice as many 0.4 and 0.7 us
// (NVFP4), 1.0 and 1.0 us (MXFP8).
constexpr int DEC_MIN_VALUES = 1024;
// Most CTAs of a shared unit: their parts are read in one go (linear 3x14336->4096, MXFP8: 15.1 us, with 9 parts 15.3;
// 19x11136->2304: 13.4 and 14.6; the other way 1x14336->1024, whose K would do for 14: 9.8 and 9.0).
constexpr int DEC_MAX_PARTS = 8;
// Half of 228 KB less the 1 KB the system keeps per CTA, so that a kernel's CTAs fit beside those of the
// kernel before it; the whole SM where that leaves fewer than three stages.
constexpr int DEC_SMEM_HALF = 113 * 1024, DEC_SMEM_FULL = 226 * 1024;
constexpr uint32_t DEC_TMEM_HALF = 256, DEC_TMEM_FULL = 512;   // likewise
// TMEM columns: accumulators (at most 160, twice where they fit), then as many sets of scales of A and B as fit, used in
// turn (at least two): a step's scales may be written while the MMAs of that many steps less one are pending.
constexpr int SPLIT_THREADS = 1024;          // at most
// Binades from a row's largest NVFP4 block scale, 2^8, to the smallest number of UE4M3, 2^-9.
constexpr int NV_SPAN = 17;
constexpr int LIFT_THREADS = 128;

enum DecMode { DEC_UP = 0, DEC_DOWN = 1, DEC_LINEAR = 2 };
enum DecFmt { DEC_MX = 0, DEC_NV = 1 };

// Warp 0 copies, warp 1 issues MMAs, then come the warps that write the columns' scales (they take turns), and four
// for the epilogue.  Linears have three for the scales (NVFP4, 61x4096->28672: 21.7 us, 25.8 with two; elsewhere the
// same); UP needs an even number, and its registers leave room for two.
constexpr int dec_scale_warps(int mode) { return mode == DEC_LINEAR ? 3 : 2; }
constexpr int dec_threads(int mode) { return 32 * (2 + dec_scale_warps(mode) + 4); }

// Columns per activation row: E4M3 pieces of a bf16 (2) or fp32 (3) value, or base-8 digits (5).
constexpr int dec_pieces(int fmt, int mode) { return fmt == DEC_NV ? 5 : mode == DEC_DOWN ? 3 : 2; }
constexpr int dec_step_values(int fmt) { return fmt == DEC_NV ? 256 : 128; }
constexpr int dec_atoms(int fmt) { return fmt == DEC_NV ? 4 : 1; }          // scale atoms per 128 rows and step
constexpr int dec_exp_bytes(int fmt) { return fmt == DEC_NV ? 16 : 4; }     // blocks of one row and step
// Most rows of a unit.  LINEAR: one accumulator of at most 64 (MXFP8) or 160 (NVFP4) columns; more tokens come in two
// chunks (one chunk of 64 measured the same with MXFP8).  MoE: two accumulators of at most 80 (an expert with more
// tokens gives several units).  Units of the same weights read them side by side, from L2.
constexpr int dec_group(int fmt, int mode) { return fmt == DEC_NV && mode != DEC_LINEAR ? 16 : 32; }

// Shared memory of one CTA (byte offsets from a 1024-byte boundary); the weight ring is at 0.
struct DecLayout {
  int stages, smem;
  int b_stage, sfb_stage;
  int b, sfa, sfb, bars, misc;
  int n_max;             // most columns of one accumulator (UP: the second one starts there)
  int acc_two;           // 1: two buffers of accumulators, for alternate units
  int sf_col, sf_cols, sf_sets;   // TMEM: first column of the scale sets, columns per set, sets
  uint32_t tmem_cols;
};

// Activations as columns of the MMA.  Row r * P + q of `codes` holds piece q of row r: 128 code bytes per K step.
struct DecOperand {
  uint8_t* codes;   // [rows * P][steps * 128]
  uint8_t* exps;    // [rows][steps][4 | 16]: exponent + 127 of every 32 | 16 values (255: not finite)
  int* top;         // [rows] largest exponent of the row (NVFP4)
  int* low;         // [rows] smallest exponent of the row's blocks but those of zeros (NVFP4, h)
};

struct DecParams {
  DecLayout L;
  DecOperand in;          // UP, LINEAR: x;  DOWN: h
  DecOperand h;           // UP: where h goes
  int h_steps;            // UP: K steps of h
  const uint8_t* w_sf;
  const float* w_amax;    // NVFP4
  const int32_t* experts; // [T, k]
  const float* gate;      // UP: [pairs] routing weights
  uint16_t* out;          // LINEAR: [T, N]
  float* y;               // DOWN: [pairs, H]
  uint32_t* err;
  float* part;            // partial sums: part_slot floats per CTA
  int part_slot;
  int* counters;          // [units][4] of units shared by several CTAs: how many are done with a quarter of the rows
  int T, k, E;
  int K;                  // contraction length of one weight row
  int steps;              // its K steps
  int kt;                 // its scale atoms per 128-row tile
  int tiles;              // 128-row tiles (of F, H or N)
  int max_active;         // most list entries (see the routing)
  int chunks, per_chunk;  // LINEAR: token chunks, tokens per chunk
  int box_rows;           // activation rows in a box of columns
  uint64_t timeout_ns, drain_ns;
};

__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// Wait for the grids this one depends on; what they wrote may then be read, by bulk copies too.
__device__ __forceinline__ void pdl_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("fence.proxy.async.global;" ::: "memory");
}
// Copies of weights: read once, so first to leave the L2 (activations, workspace and instructions stay).
__device__ __forceinline__ uint64_t evict_first() {
  uint64_t policy;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}
__device__ __forceinline__ void tma_load_weights(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4}], "
      "[%2], %5;" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void bulk_load_weights(void* dst, const void* src, uint32_t bytes, uint64_t* bar,
                                                  uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
// One lane of the (converged) warp.  The compiler knows that a branch on it holds one thread, and issues
// copies and MMAs there directly; behind `lane == 0` it wraps each of them in a loop over the lanes.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
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

// Four values' E2M1 codes, the first in the lowest nibble.
__device__ __forceinline__ uint32_t e2m1x4_f2(uint64_t v, uint64_t w) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "mov.b32 %0, {a, b, a, b};\n\t}"
      : "=r"(r)
      : "f"(f2_lo(v)), "f"(f2_hi(v)), "f"(f2_lo(w)), "f"(f2_hi(w)));
  return r & 0xFFFFu;
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
  if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;   // mostly: one instruction for the warp
  int ok = 1;
  if (lane == 0) ok = dec_wait(bar, parity, abort, p, err_bit) ? 1 : 0;
  return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
}

// floor(log2) of a block's largest magnitude from its float bits (128: not finite), kept where the
// scales used below stay representable: blocks under 2^-100 count as 2^-100.
__device__ __forceinline__ int block_exponent(uint32_t abs_bits) {
  return max(static_cast<int>(abs_bits >> 23) - 127, -100);
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// Multiplier that takes a block's largest magnitude into [128, 256) (MXFP8) or [2, 4) (NVFP4).
template <int FMT>
__device__ __forceinline__ float block_multiplier(int eb) {
  return pow2f((FMT == DEC_NV ? 1 : 7) - min(eb, 127));
}
// One step of the decomposition: the next piece of a pair of scaled values, and what is left of them
// for the following piece.  MXFP8: the leading 4 bits of the significand, or (last) all of it, rounded
// by the conversion; NVFP4: the nearest integer (adding and subtracting 1.5 * 2^23 rounds to it).
template <int FMT, bool LAST>
__device__ __forceinline__ uint64_t next_piece(uint64_t& r) {
  if constexpr (FMT == DEC_MX) {
    if constexpr (LAST) return r;
    const uint64_t top = r & 0xFFF00000FFF00000ull;
    r = f2_mul(f2_fma(top, f2_pack(-1.0f, -1.0f), r), f2_pack(16.0f, 16.0f));
    return top;
  } else {
    const uint64_t n = f2_add(f2_add(r, f2_pack(12582912.0f, 12582912.0f)), f2_pack(-12582912.0f, -12582912.0f));
    if constexpr (!LAST) r = f2_fma(n, f2_pack(-8.0f, -8.0f), f2_mul(r, f2_pack(8.0f, 8.0f)));
    return n;
  }
}

// Sum over a value's columns, smallest piece first; a digit's place is 1/8 of the one before.
template <int FMT, int P>
__device__ __forceinline__ float sum_pieces(const uint32_t* d) {
  float x = __uint_as_float(d[P - 1]);
#pragma unroll
  for (int z = P - 2; z >= 0; --z)
    x = FMT == DEC_NV ? fmaf(x, 0.125f, __uint_as_float(d[z])) : x + __uint_as_float(d[z]);
  return x;
}

// The code bytes of the next piece of eight (MXFP8) or sixteen (NVFP4) scaled values.
template <int FMT, bool LAST>
__device__ __forceinline__ uint2 next_codes(uint64_t (&r)[FMT == DEC_NV ? 8 : 4]) {
  constexpr int N = FMT == DEC_NV ? 8 : 4;
  uint64_t n[N];
#pragma unroll
  for (int i = 0; i < N; ++i) n[i] = next_piece<FMT, LAST>(r[i]);
  uint2 code;
  if constexpr (FMT == DEC_MX) {
    code.x = e4m3x2_f2(n[0]) | (e4m3x2_f2(n[1]) << 16);
    code.y = e4m3x2_f2(n[2]) | (e4m3x2_f2(n[3]) << 16);
  } else {
    code.x = e2m1x8(f2_lo(n[0]), f2_hi(n[0]), f2_lo(n[1]), f2_hi(n[1]), f2_lo(n[2]), f2_hi(n[2]), f2_lo(n[3]),
                    f2_hi(n[3]));
    code.y = e2m1x8(f2_lo(n[4]), f2_hi(n[4]), f2_lo(n[5]), f2_hi(n[5]), f2_lo(n[6]), f2_hi(n[6]), f2_lo(n[7]),
                    f2_hi(n[7]));
  }
  return code;
}

// x (bf16 [T, K]) -> columns; a thread takes 8 values (MXFP8, four threads a block) or 16 (NVFP4, one block)
// at a time, 8 code bytes either way.  It also prepares the call's bookkeeping: the error word, the range
// check of the experts' ids, the row exponents of h and the counters.
//   BY_PAIR  one CTA per choice (t, j), which finds the choice's pair as the weight kernels' routing numbers
//            them, writes its token's columns there and the pair's routing weight (a token that lists an expert
//            more than once is one pair with the sum of the weights); a choice that is dropped or repeats an
//            earlier one has none.
//   else     one CTA per token.
// Latency-bound (a token is a few KB): what matters is that the weight kernel's copies start meanwhile.
struct SplitParams {
  const uint16_t* x;
  DecOperand o;
  uint32_t* err;
  const int32_t* experts;
  const float* gates;
  float* gate;            // [pairs]
  int* row_of;            // [T, k] pair of every choice (-1: none)
  int *h_top, *h_low;
  int* counters;
  int T, K, steps, n_ids, E, k, n_top, n_counters;
};
template <int FMT, bool BY_PAIR>
__global__ void __launch_bounds__(SPLIT_THREADS) k_split_x(const SplitParams p) {
  constexpr int P = dec_pieces(FMT, DEC_LINEAR), EB = dec_exp_bytes(FMT);
  constexpr int VALS = FMT == DEC_NV ? 16 : 8;   // 16 groups per step
  __shared__ int s_top, s_row;
  __shared__ int s_ids[BY_PAIR ? DEC_MAX_TOKENS * DEC_MAX_K : 1];
  pdl_wait();
  const int b = blockIdx.x, t = BY_PAIR ? b / p.k : b, tid = threadIdx.x;
  if (tid == 0) {
    s_top = -128;
    s_row = 0;
  }
  pdl_launch_dependents();   // everything before this call in the stream is complete
  // this thread's first values: on their way while the pair is looked up
  const int groups = p.K / VALS;
  uint4 ahead[VALS / 8];
#pragma unroll
  for (int i = 0; i < VALS / 8; ++i)
    ahead[i] = tid < groups
                   ? __ldg(reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(t) * p.K + tid * VALS) + i)
                   : make_uint4(0u, 0u, 0u, 0u);
  int bad = 0;
  if constexpr (BY_PAIR)
    for (int i = tid; i < p.n_ids; i += blockDim.x) {
      const int e = __ldg(p.experts + i);
      s_ids[i] = e;
      bad |= e >= p.E ? 1 : 0;
    }
  bad = __syncthreads_or(bad);
  if (b == 0 && tid == 0) *p.err = bad ? ERR_EXPERT_RANGE : 0u;
  for (int i = b * blockDim.x + tid; i < p.n_top; i += gridDim.x * blockDim.x) {
    p.h_top[i] = -128;
    p.h_low[i] = 128;
  }
  for (int i = b * blockDim.x + tid; i < p.n_counters; i += gridDim.x * blockDim.x) p.counters[i] = 0;

  int dst = t;   // row of the operand
  if constexpr (BY_PAIR) {
    // pairs of lower experts, and of this expert with lower tokens
    const int e = s_ids[b];
    bool none = e < 0 || e >= p.E;
    for (int j = t * p.k; j < b; ++j) none |= s_ids[j] == e;
    int below = 0;
    if (!none)
      for (int i = tid; i < p.n_ids; i += blockDim.x) {
        const int o = s_ids[i], ot = i / p.k;
        bool first = o >= 0 && (o < e || (o == e && ot < t));
        for (int j = ot * p.k; first && j < i; ++j) first = s_ids[j] != o;
        below += first ? 1 : 0;
      }
    below = __reduce_add_sync(0xFFFFFFFFu, below);
    if ((tid & 31) == 0 && below != 0) atomicAdd(&s_row, below);
    __syncthreads();
    dst = s_row;
    if (tid == 0) {
      p.row_of[b] = none ? -1 : dst;
      float g = 0.0f;
      for (int j = b; !none && j < (t + 1) * p.k; ++j)
        if (s_ids[j] == e) g += p.gates != nullptr ? __ldg(p.gates + j) : 1.0f;
      if (!none) p.gate[dst] = g;
    }
    if (none) return;
  }

  // bf16 values of this thread's group gi, and their largest magnitude's bits
  auto load = [&](int g0, uint4 (&w)[VALS / 8]) {
    const int gi = g0 + tid;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < VALS / 8; ++i) {
      w[i] = g0 == 0 ? ahead[i]
             : gi < groups ? __ldg(reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(t) * p.K + gi * VALS) + i)
                           : make_uint4(0u, 0u, 0u, 0u);
      m = __vmaxu2(m, __vmaxu2(__vmaxu2(w[i].x & 0x7FFF7FFFu, w[i].y & 0x7FFF7FFFu),
                               __vmaxu2(w[i].z & 0x7FFF7FFFu, w[i].w & 0x7FFF7FFFu)));
    }
    return max(m & 0xFFFFu, m >> 16) << 16;
  };
  // NVFP4: the row's largest exponent comes first, since the blocks' scales reach NV_SPAN binades below it; a smaller
  // block is written under the smallest scale, in its lower digits.
  int lowest = -128;
  if constexpr (FMT == DEC_NV) {
    int top = -128;
    uint4 w[VALS / 8];
    for (int g0 = 0; g0 < groups; g0 += blockDim.x) top = max(top, block_exponent(load(g0, w)));
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if ((tid & 31) == 0) atomicMax(&s_top, top);
    __syncthreads();
    lowest = s_top - NV_SPAN;
    if (tid == 0) p.o.top[dst] = s_top;
  }
  for (int g0 = 0; g0 < groups; g0 += blockDim.x) {
    const int gi = g0 + tid;
    const bool in = gi < groups;   // K % 128 == 0: whole blocks, and the four threads of one agree
    const int step = gi >> 4, g = gi & 15;
    uint4 w[VALS / 8];
    uint32_t m = load(g0, w);
    if constexpr (FMT == DEC_MX) {
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    }
    if (!in) continue;
    const int eb = max(block_exponent(m), lowest);
    if (FMT == DEC_NV || (g & 3) == 0)
      p.o.exps[(static_cast<int64_t>(dst) * p.steps + step) * EB + (FMT == DEC_NV ? g : g >> 2)] =
          static_cast<uint8_t>(eb + 127);
    const uint64_t inv2 = f2_pack(block_multiplier<FMT>(eb), block_multiplier<FMT>(eb));
    uint64_t r[VALS / 2];
#pragma unroll
    for (int i = 0; i < VALS / 8; ++i) {
      r[4 * i] = f2_mul(f2_pack(bf16_lo(w[i].x), bf16_hi(w[i].x)), inv2);
      r[4 * i + 1] = f2_mul(f2_pack(bf16_lo(w[i].y), bf16_hi(w[i].y)), inv2);
      r[4 * i + 2] = f2_mul(f2_pack(bf16_lo(w[i].z), bf16_hi(w[i].z)), inv2);
      r[4 * i + 3] = f2_mul(f2_pack(bf16_lo(w[i].w), bf16_hi(w[i].w)), inv2);
    }
#pragma unroll
    for (int q = 0; q < P; ++q) {
      const uint2 code = q + 1 < P ? next_codes<FMT, false>(r) : next_codes<FMT, true>(r);
      *reinterpret_cast<uint2*>(p.o.codes + (static_cast<int64_t>(dst) * P + q) * p.steps * 128 + gi * 8) = code;
    }
  }
}

// The scale words of one activation row and K step for its P columns, from its blocks' exponents.
//   MXFP8  word of piece q: UE8M0 2^(e - 7 - 4 q) per block.
//   NVFP4  one word per MMA, the same for all digits: UE4M3 2^(8 + e - top) per block (e >= top - NV_SPAN).
// Blocks that are not finite get a NaN scale.
// (Plain arithmetic: the byte-wise intrinsics are chains of instructions, 0.4 us a step for a warp alone.)
__device__ __forceinline__ uint32_t mx_scales(uint32_t e4, int q) {
  const uint32_t ones = ((e4 & 0x7F7F7F7Fu) + 0x01010101u) & e4 & 0x80808080u;   // the top bit of a byte of ones
  return (e4 - (0x07070707u + 0x04040404u * static_cast<uint32_t>(q))) | ((ones >> 7) * 0xFFu);   // e4 >= 27: no borrow
}
__device__ __forceinline__ uint32_t nv_scales(uint32_t e4, int top) {
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = static_cast<int>((e4 >> (8 * i)) & 0xFFu);
    v[i] = __uint_as_float(e == 255 ? 0x7FC00000u : static_cast<uint32_t>(max(e - top + 8, 0)) << 23);
  }
  return e4m3x2_f2(f2_pack(v[0], v[1])) | (e4m3x2_f2(f2_pack(v[2], v[3])) << 16);
}

// The K steps of all units (128-row tiles; MoE: of a chosen expert, for a group of its tokens) form one
// sequence; a CTA runs through a part of one unit and then through whole ones.  Where several CTAs share a
// unit, whoever finishes last sums the parts, in their order (the result does not depend on who it is).
template <int FMT, int MODE>
__global__ void __launch_bounds__(dec_threads(MODE), 2) k_decode(const __grid_constant__ CUtensorMap tm_w,
                                                           const __grid_constant__ CUtensorMap tm_x, const DecParams p) {
  constexpr int P = dec_pieces(FMT, MODE);
  constexpr int ATOMS = dec_atoms(FMT), EB = dec_exp_bytes(FMT);
  constexpr bool UP = MODE == DEC_UP, MOE = MODE != DEC_LINEAR;
  constexpr int ACCS = UP ? 2 : 1, MIN_STEPS = DEC_MIN_VALUES / dec_step_values(FMT);
  constexpr int THREADS = dec_threads(MODE), SCALE_WARPS = dec_scale_warps(MODE), FIRST_EPI_WARP = 2 + SCALE_WARPS;
  constexpr int GROUP = dec_group(FMT, MODE);
  static_assert(GROUP <= 32, "a lane per row");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const DecLayout& L = p.L;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L.bars);   // the copies landed, the columns' scales are in place
  uint64_t* empty = full + DEC_MAX_STAGES;                        // the MMAs have read the stage
  uint64_t* acc_full = empty + DEC_MAX_STAGES;                    // [2] this CTA's part of a unit is complete in TMEM
  uint64_t* acc_empty = acc_full + 2;                             // [2] the epilogue has read it
  uint64_t* drained = acc_empty + 2;                              // [4] MMA warp, scale warps: nothing in flight
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drained + 4);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* s_nact = reinterpret_cast<int*>(tmem_holder + 2);
  // MoE: tokens that chose the expert [E]; then the list of groups of tokens: expert, first pair, pairs
  uint64_t* s_mask = reinterpret_cast<uint64_t*>(smem + L.misc);
  int* s_act_e = reinterpret_cast<int*>(s_mask + p.E);
  int* s_act_row = s_act_e + p.max_active;
  int* s_act_n = s_act_row + p.max_active;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int chunk = static_cast<int>(blockIdx.x) % p.chunks;   // LINEAR: the chunks' CTAs run side by side

  if (MOE && tid == 0) pdl_launch_dependents();
  if (tid == 0) {
    for (int s = 0; s < L.stages; ++s) {
      mbar_init(&full[s], 2);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], 4);
    }
    for (int s = 0; s < 1 + SCALE_WARPS; ++s) mbar_init(&drained[s], 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, L.tmem_cols);
    tmem_relinquish();
  }

  // ---- routing: which tokens chose which expert, and the list of chosen experts ----
  if constexpr (MOE) {
    const int ids = p.T * p.k;
    int e = tid < ids ? __ldg(p.experts + tid) : -1;   // on its way meanwhile
    for (int z = tid; z < p.E; z += THREADS) s_mask[z] = 0;
    __syncthreads();
    for (int i = tid; i < ids; i += THREADS, e = i < ids ? __ldg(p.experts + i) : -1) {
      const int t = i / p.k;
      if (e >= 0 && e < p.E) atomicOr(reinterpret_cast<uint32_t*>(&s_mask[e]) + (t >> 5), 1u << (t & 31));
    }
    __syncthreads();
    if (warp == 0) {
      int n = 0, rows = 0;
      for (int base = 0; base < p.E; base += 32) {
        const int pop = base + lane < p.E ? __popcll(s_mask[base + lane]) : 0;
        const int groups = (pop + GROUP - 1) / GROUP;
        if (__ballot_sync(0xFFFFFFFFu, pop != 0) == 0) continue;
        int incl = pop | (groups << 16);   // two running sums in one word: pairs and groups are below 2^12
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
          if (lane >= d) incl += o;
        }
        const int pos = n + (incl >> 16) - groups, row = rows + (incl & 0xFFFF) - pop;
        for (int g = 0; g < groups; ++g) {
          s_act_e[pos + g] = base + lane;
          s_act_row[pos + g] = row + g * GROUP;
          s_act_n[pos + g] = min(GROUP, pop - g * GROUP);
        }
        const int last = __shfl_sync(0xFFFFFFFFu, incl, 31);
        n += last >> 16;
        rows += last & 0xFFFF;
      }
      if (lane == 0) *s_nact = n;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  // ---- this CTA's piece of the sequence ----
  const int su = UP ? 2 * p.steps : p.steps;                    // steps of a unit
  const int units = MOE ? *s_nact * p.tiles : p.tiles;
  // Every CTA takes the same number of whole units; the units left over are shared, each by as many CTAs as fit
  // (and find MIN_STEPS steps).  The share comes first, so that adding its parts up is hidden.  per_unit is rounded
  // down: 224 units and no whole ones leave 80 of 304 CTAs without work.  (Dealing the left-over steps out evenly, with
  // two parts of units in a CTA, measured 5-15% slower while parts were added one by one; not measured again since.)
  const int slots = static_cast<int>(gridDim.x) / p.chunks, cta = static_cast<int>(blockIdx.x) / p.chunks;
  const int whole = units / slots, shared = units - whole * slots;
  // CTAs of a shared unit
  const int per_unit = shared == 0 ? 1 : max(1, min(DEC_MAX_PARTS, min(slots / shared, su / MIN_STEPS)));
  // Place in the sequence: list entry, 128-row tile, K step, accumulator.  Divisions only here.
  struct Place {
    int a, tile, f, acc;
  };
  auto unit_at = [&](int u) { return Place{u / p.tiles, u % p.tiles, 0, 0}; };
  const Place first_whole = unit_at(cta * whole);
  Place first = first_whole;
  int n_share = 0;   // this CTA's steps of its share
  if (cta < shared * per_unit) {
    const int u = cta / per_unit, o = cta - u * per_unit, r = su * o / per_unit;
    n_share = su * (o + 1) / per_unit - r;
    first = unit_at(slots * whole + u);
    first.f = UP ? r >> 1 : r;
    first.acc = UP ? r & 1 : 0;
  }
  const int n_steps = n_share + whole * su;
  // Activation rows of list entry a (LINEAR: of the chunk), and the columns of its MMA.
  auto rows_of = [&](int a) { return MOE ? s_act_n[a] : min(p.per_chunk, p.T - chunk * p.per_chunk); };
  auto first_row = [&](int a) { return MOE ? s_act_row[a] : chunk * p.per_chunk; };
  auto mma_columns = [&](int a) { return (P * rows_of(a) + 15) & ~15; };
  auto advance = [&](Place& q, int i) {   // from step i to the next
    if (i + 1 == n_share) {
      q = first_whole;
      return;
    }
    if constexpr (UP) q.acc ^= 1;
    if (q.acc != 0 || ++q.f < p.steps) return;
    q.f = 0;
    if (++q.tile < p.tiles) return;
    q.tile = 0;
    ++q.a;
  };
  // Stage of the ring, and the parity of its current use.
  struct Ring {
    int slot;
    uint32_t phase;
  };
  auto next_stage = [&](Ring& r) {
    if (++r.slot == L.stages) {
      r.slot = 0;
      r.phase ^= 1u;
    }
  };

  if (warp == 0) {
    // ---------------- copies (one lane) ----------------
    if (elect_one()) {
      const uint64_t policy = evict_first();
      // of the unit at hand: its first weight row and scale atoms per accumulator, and its first column
      int unit_a = -1, unit_tile = -1, row[ACCS], column = 0;
      const uint8_t* sf[ACCS];
      // First the ring is filled with weights, before waiting for the activations the previous kernel writes; then
      // come those stages' columns, and all that is left.
      const int fill = min(n_steps, L.stages);
      int issued = 0;
      Ring r{0, 0};
#pragma unroll 1
      for (int pass = 0; pass < 2; ++pass) {
        if (pass == 1) pdl_wait();
        const int end = pass == 0 ? fill : n_steps;
        Place q = first;
        r = Ring{0, 0};
#pragma unroll 1
        for (issued = 0; issued < end; advance(q, issued), ++issued, next_stage(r)) {
          const bool refill = issued >= fill;
          if (refill && !dec_wait(&empty[r.slot], r.phase ^ 1u, abort_flag, p, ERR_TIMEOUT_PRODUCER)) break;
          if (q.tile != unit_tile || q.a != unit_a) {
            unit_a = q.a;
            unit_tile = q.tile;
            column = first_row(q.a) * P;
#pragma unroll
            for (int c = 0; c < ACCS; ++c) {
              row[c] = q.tile * 128;
              if constexpr (MOE) row[c] += (s_act_e[q.a] * ACCS + c) * (p.tiles * 128);
              sf[c] = p.w_sf + static_cast<int64_t>(row[c] >> 7) * p.kt * 512;
            }
          }
          const bool up = UP && q.acc != 0;
          if (pass == 0 || refill) {
            mbar_arrive_expect_tx(&full[r.slot], DEC_A_STAGE + ATOMS * 512 + p.box_rows * P * 128);
            tma_load_weights(smem + r.slot * DEC_A_STAGE, &tm_w, &full[r.slot], q.f * 128, up ? row[ACCS - 1] : row[0],
                             policy);
            bulk_load_weights(smem + L.sfa + r.slot * ATOMS * 512, (up ? sf[ACCS - 1] : sf[0]) + q.f * ATOMS * 512,
                              ATOMS * 512, &full[r.slot], policy);
          }
          // the unit's columns and whatever follows them: a box has a fixed height
          if (pass == 1) tma_load_2d(smem + L.b + r.slot * L.b_stage, &tm_x, &full[r.slot], q.f * 128, column);
        }
      }
      // every copy must have landed before the CTA may exit; after a timeout elsewhere the barriers may lack
      // their other arrival, and one full drain wait is enough for all the copies
      Ring e = issued < L.stages ? Ring{0, 0} : Ring{r.slot, r.phase ^ 1u};
      for (int z = min(issued, L.stages); z > 0; --z, next_stage(e))
        if (!mbar_wait_bounded(&full[e.slot], e.phase, nullptr, p.drain_ns)) {
          atomicOr(p.err, ERR_TIMEOUT_DRAIN);
          break;
        }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- scale copies and MMAs (one lane) ----------------
    if (elect_one()) {
      // descriptors of stage 0: addresses are in units of 16 bytes in their low bits
      const uint64_t desc_a = sdesc_kmajor_sw128(smem_u32(smem)), desc_b = sdesc_kmajor_sw128(smem_u32(smem + L.b));
      const uint64_t desc_sfa = sdesc_sf_atom(smem_u32(smem + L.sfa));
      bool ok = true, any = false;
      pdl_wait();   // the columns come after it anyway: the limits of the waits start here
      Ring r{0, 0};
      int i = 0, set = 0;
      Place q = first;
      for (int seg = 0; ok && i < n_steps; ++seg) {
        const int a = q.a, tile = q.tile;
        const int n_mma = mma_columns(a), nat = (n_mma + 127) >> 7;
        const uint32_t idesc = FMT == DEC_NV ? idesc_nvf4(128, n_mma) : idesc_mxf8_e4m3(128, n_mma);
        uint32_t started = 0;   // accumulators that hold something
        const int buf = seg & L.acc_two;
        if (seg > L.acc_two &&
            !dec_wait(&acc_empty[buf], ((seg >> L.acc_two) - 1) & 1, abort_flag, p, ERR_TIMEOUT_MMA))
          break;
        tc_fence_after();
        for (; i < n_steps && q.a == a && q.tile == tile; advance(q, i), ++i, next_stage(r)) {
          const int slot = r.slot;
          if (!dec_wait(&full[slot], r.phase, abort_flag, p, ERR_TIMEOUT_MMA)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t da = desc_a + slot * (DEC_A_STAGE >> 4), db = desc_b + slot * (L.b_stage >> 4);
          const uint64_t dsa = desc_sfa + slot * (ATOMS * 32);
          const uint32_t t_sfa = tmem + L.sf_col + set * L.sf_cols, t_sfb = t_sfa + 4 * ATOMS;
          if (++set == L.sf_sets) set = 0;
          const uint32_t d = tmem + (buf * ACCS + q.acc) * L.n_max;
#pragma unroll
          for (int m = 0; m < ATOMS; ++m) tc_copy_sf(t_sfa + 4 * m, dsa + 32 * m);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t add = ((started >> q.acc) & 1u) | (k != 0 ? 1u : 0u);
            if constexpr (FMT == DEC_NV)
              tc_mma_nvf4(d, da + 2 * k, db + 2 * k, idesc, t_sfa + 4 * k, t_sfb + 4 * nat * k, add);
            else
              tc_mma_mxf8(d, da + 2 * k, db + 2 * k, idesc_with_sf_id(idesc, k), t_sfa, t_sfb, add);
          }
          started |= 1u << q.acc;
          tc_commit(&empty[slot]);
          any = true;
        }
        if (ok) tc_commit(&acc_full[buf]);
      }
      if (any) {
        tc_commit(drained);
        if (!mbar_wait_bounded(drained, 0, nullptr, p.drain_ns)) atomicOr(p.err, ERR_TIMEOUT_DRAIN);
      }
    }
    __syncwarp();
  } else if (warp < FIRST_EPI_WARP) {
    // ---------------- the columns' scales: warp cw takes every SCALE_WARPS-th step, from cw ----------------
    // It writes them to shared memory, has them copied to the step's set in TMEM (here, not by the MMA thread,
    // whose time per step is what limits a CTA), and the copies' completion counts on `full`.
    // The set (and the stage) must have been read by step i - sf_sets.  Fewer warps than stages: when a warp
    // waits for that step, the use of its stage before it is known to be over, as a wait by parity requires.
    const int cw = warp - 2;
    // MXFP8, and NVFP4 with more than eight rows: lane = row, all its words; NVFP4 with up to eight:
    // lane = (word, row), one of the row's four words.
    // One warp does all of a step, so the code between two steps is kept short, and nothing touches a loaded value
    // before the step it is for.
    struct Scales {
      uint32_t e[ATOMS];
      int c, top, n, nat, f;   // row of the unit (lanes past the last: none) and its reference, rows, atoms per MMA
      bool spread;
    };
    int entry = -1;
    const uint8_t* src = nullptr;   // of this lane's row
    Scales cur{}, next{};
    auto load = [&](const Place& q, Scales& v) {
      if (q.a != entry) {
        entry = q.a;
        v.n = rows_of(q.a);
        v.nat = (mma_columns(q.a) + 127) >> 7;
        v.spread = FMT == DEC_NV && v.n <= 8;
        v.c = v.spread ? lane & 7 : lane;
        const int row = first_row(q.a) + min(v.c, v.n - 1);
        if constexpr (FMT == DEC_NV) v.top = p.in.top[row];
        src = p.in.exps + static_cast<int64_t>(row) * p.steps * EB + (v.spread ? (lane >> 3) * 4 : 0);
      }
      v.f = q.f;
      const uint8_t* at = src + q.f * EB;
      if constexpr (FMT == DEC_NV) {
        if (v.spread) {
          v.e[0] = *reinterpret_cast<const uint32_t*>(at);
        } else {
          const uint4 w = *reinterpret_cast<const uint4*>(at);
          v.e[0] = w.x; v.e[1] = w.y; v.e[2] = w.z; v.e[3] = w.w;
        }
      } else {
        v.e[0] = *reinterpret_cast<const uint32_t*>(at);
      }
    };
    // place of a column's word of the first atom, from the start of the step's scales
    auto word = [](int col) { return (col >> 7) * 512 + (col & 31) * 16 + ((col >> 5) & 3) * 4; };
    Place q = first;
#pragma unroll 1
    for (int z = 0; z < cw; ++z) advance(q, z);
    pdl_wait();
    if (cw < n_steps) load(q, cur);
    int slot = cw, set = cw % L.sf_sets;
    const int set_next = SCALE_WARPS % L.sf_sets;
    Ring read{cw >= L.sf_sets ? cw - L.sf_sets : 0, 0};   // stage of step i - sf_sets
    const uint64_t desc_sfb = sdesc_sf_atom(smem_u32(smem + L.sfb));
    for (int i = cw; i < n_steps; i += SCALE_WARPS) {
      next = cur;
      if (i + SCALE_WARPS < n_steps) {
        // mostly on along K, for the same accumulator
        static_assert(SCALE_WARPS % ACCS == 0, "same accumulator");
        if (q.f + SCALE_WARPS / ACCS < p.steps && (i >= n_share || i + SCALE_WARPS < n_share)) {
          q.f += SCALE_WARPS / ACCS;
        } else {
#pragma unroll 1
          for (int z = 0; z < SCALE_WARPS; ++z) advance(q, i + z);
        }
        load(q, next);
      }
      uint32_t w[ATOMS];
      if constexpr (FMT == DEC_NV) {
        // words past the row's end count as zeros
        w[0] = nv_scales((cur.f * 4 + (cur.spread ? lane >> 3 : 0)) * 64 < p.K ? cur.e[0] : 0u, cur.top);
        if (!cur.spread)
#pragma unroll
          for (int m = 1; m < 4; ++m) w[m] = nv_scales((cur.f * 4 + m) * 64 < p.K ? cur.e[m] : 0u, cur.top);
      } else {
        w[0] = cur.e[0];
      }
      if (i >= L.sf_sets) {
        if (!dec_warp_wait(&empty[read.slot], read.phase, abort_flag, p, ERR_TIMEOUT_SF, lane)) break;
        tc_fence_after();   // the copies to the set below come after the MMAs that read it
#pragma unroll
        for (int z = 0; z < SCALE_WARPS; ++z) next_stage(read);
      } else if (i + SCALE_WARPS >= L.sf_sets) {
        read = Ring{i + SCALE_WARPS - L.sf_sets, 0};   // of the next step of this warp
      }
      uint8_t* sf = smem + L.sfb + slot * L.sfb_stage;
      if (cur.c < cur.n) {
#pragma unroll
        for (int d = 0; d < P; ++d) {
          uint8_t* dst = sf + word(cur.c * P + d);
          if constexpr (FMT == DEC_MX) {
            *reinterpret_cast<uint32_t*>(dst) = mx_scales(w[0], d);
          } else if (cur.spread) {
            *reinterpret_cast<uint32_t*>(dst + (lane >> 3) * 512) = w[0];
          } else {
#pragma unroll
            for (int m = 0; m < 4; ++m) *reinterpret_cast<uint32_t*>(dst + m * cur.nat * 512) = w[m];
          }
        }
      }
      fence_proxy_async_smem();   // the tensor core reads these bytes through the async proxy
      __syncwarp();
      if (elect_one()) {
        const uint64_t dsb = desc_sfb + slot * (L.sfb_stage >> 4);
        const uint32_t t_sfb = tmem + L.sf_col + set * L.sf_cols + 4 * ATOMS;
        for (int m = 0; m < ATOMS * cur.nat; ++m) tc_copy_sf(t_sfb + 4 * m, dsb + 32 * m);
        tc_commit(&full[slot]);
      }
      __syncwarp();
      cur = next;
      slot = slot + SCALE_WARPS < L.stages ? slot + SCALE_WARPS : slot + SCALE_WARPS - L.stages;
      set += set_next;
      if (set >= L.sf_sets) set -= L.sf_sets;
    }
    if (cw < n_steps && elect_one()) {
      tc_commit(&drained[1 + cw]);
      if (!mbar_wait_bounded(&drained[1 + cw], 0, nullptr, p.drain_ns)) atomicOr(p.err, ERR_TIMEOUT_DRAIN);
    }
    __syncwarp();
  } else {
    // ---------------- epilogue ----------------
    pdl_wait();
    const int quarter = warp & 3, row = quarter * 32 + lane;
    float alpha = 1.0f;
    if constexpr (FMT == DEC_NV) alpha = 1.0f / nv_encode_scale(__ldg(p.w_amax));
    int i = 0;
    Place q = first;
    for (int seg = 0; i < n_steps; ++seg) {
      const bool share = i < n_share && per_unit > 1;
      const int u = cta / per_unit, parts = per_unit;   // if shared: which unit, how many parts
      const int n = rows_of(q.a), row0 = first_row(q.a), tile = q.tile;
      float unscale = 1.0f;   // lane c: of row c's sums
      if constexpr (FMT == DEC_NV) unscale = ldexpf(alpha, p.in.top[row0 + min(lane, n - 1)] - 9);
      // y of activation row c and this thread's weight row
      auto put = [&](int c, float v) {
        const int64_t o = static_cast<int64_t>(row0 + c) * (p.tiles * 128) + tile * 128 + row;
        if constexpr (MODE == DEC_DOWN) p.y[o] = v;
        else p.out[o] = static_cast<uint16_t>(pack_bf16x2(v, 0.0f) & 0xFFFFu);
      };
      // part o of the unit: [accumulator][activation row][128 weight rows], in the place of the CTA that has it
      auto part_of = [&](int o) {
        return p.part + static_cast<int64_t>((u * per_unit + o) * p.chunks + chunk) * p.part_slot;
      };

      const int buf = seg & L.acc_two;
      const uint32_t t_row = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + buf * ACCS * L.n_max;
      if (!dec_warp_wait(&acc_full[buf], (seg >> L.acc_two) & 1, abort_flag, p, ERR_TIMEOUT_EPILOGUE, lane)) break;
      tc_fence_after();
      float* mine = part_of(cta - u * per_unit) + row;
      int* counter = p.counters + (chunk * shared + u) * 4 + quarter;   // each warp for its 32 weight rows
      // A part of a unit is in memory; true in the warp that finds all the others there too.
      auto last_part = [&]() {
        int before = 0;
        if (lane == 0) {
          __threadfence();
          before = atomicAdd(counter, 1);
          __threadfence();
        }
        __syncwarp();
        return __shfl_sync(0xFFFFFFFFu, before, 0) == parts - 1;
      };
      auto release = [&]() {   // the next unit's MMAs may begin
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[buf]);
      };
      if constexpr (!UP) {
#pragma unroll 1
        for (int c0 = 0; c0 < n; c0 += 4) {
          constexpr int LD = (4 * P + 7) / 8;
          uint32_t d[8 * LD];
#pragma unroll
          for (int z = 0; z < LD; ++z) tmem_ld_32x32b_x8(t_row + c0 * P + z * 8, d + z * 8);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float x = sum_pieces<FMT, P>(d + j * P);
            if constexpr (FMT == DEC_NV) x *= __shfl_sync(0xFFFFFFFFu, unscale, c0 + j);
            if (c0 + j >= n) continue;
            if (share) mine[(c0 + j) * 128] = x;
            else put(c0 + j, x);
          }
        }
        release();
        // Whoever is last adds the parts up, in order.  Eight lanes take the warp's 32 weight rows of an activation row,
        // four at a time, with all parts on their way: this is a chain of trips to the L2.
        if (share && last_part()) {
          const int r4 = quarter * 32 + (lane & 7) * 4;
#pragma unroll 1
          for (int c = lane >> 3; c < n; c += 4) {
            float4 x[DEC_MAX_PARTS], sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int o = 0; o < DEC_MAX_PARTS; ++o)
              x[o] = o < parts ? __ldcg(reinterpret_cast<const float4*>(part_of(o) + c * 128 + r4))
                               : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int o = 0; o < DEC_MAX_PARTS; ++o) {
              sum.x += x[o].x;
              sum.y += x[o].y;
              sum.z += x[o].z;
              sum.w += x[o].w;
            }
            const int64_t at = static_cast<int64_t>(row0 + c) * (p.tiles * 128) + tile * 128 + r4;
            if constexpr (MODE == DEC_DOWN)
              *reinterpret_cast<float4*>(p.y + at) = sum;
            else
              *reinterpret_cast<uint2*>(p.out + at) = make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
          }
        }
      } else {
        // h from the gate and up sums, as columns of DOWN.  In the accumulators a lane has one weight row; four lanes
        // transpose their values of four activation rows, and each converts four values of one of them (a block is 16
        // or 32 lanes wide).  (Passing the sums of whole units through memory as well, to free the accumulators earlier, measured
        // the same.)  Short straight code: its first pass is fetched line by line behind the weights' stream.
        constexpr int PH = dec_pieces(FMT, DEC_DOWN), LD = (4 * P + 7) / 8;
        static_assert(MIN_STEPS >= 2, "a part of a unit holds steps of both accumulators");
        const float gates = p.gate[row0 + min(lane, n - 1)];
        const int64_t pitch = static_cast<int64_t>(p.h_steps) * 128;
        const int k0 = tile * 128 + quarter * 32 + (lane & ~3);   // of this lane's four values
#pragma unroll 1
        for (int phase = share ? 0 : 1; phase < 2; ++phase) {
          if (phase == 1 && share && !last_part()) break;
#pragma unroll 1
          for (int c0 = 0; c0 < n; c0 += 4) {
            float v[2][4];   // [accumulator][row]
            if (phase == 0 || !share) {
              uint32_t d[2][8 * LD];
#pragma unroll
              for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int z = 0; z < LD; ++z) tmem_ld_32x32b_x8(t_row + b * L.n_max + c0 * P + z * 8, d[b] + z * 8);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float scale = FMT == DEC_NV ? __shfl_sync(0xFFFFFFFFu, unscale, (c0 + j) & 31) : 1.0f;
#pragma unroll
                for (int b = 0; b < 2; ++b) v[b][j] = sum_pieces<FMT, P>(d[b] + j * P) * scale;
              }
              if (phase == 0) {
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    if (c0 + j < n) mine[(b * n + c0 + j) * 128] = v[b][j];
                continue;
              }
              // lane l of four keeps row c0 + l, values k0 .. k0 + 3
#pragma unroll
              for (int z = 1; z < 4; z *= 2) {
                const bool up = (lane & z) != 0;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    if ((j & z) == 0) {
                      const float other = __shfl_xor_sync(0xFFFFFFFFu, up ? v[b][j] : v[b][j | z], z);
                      v[b][j] = up ? other : v[b][j];
                      v[b][j | z] = up ? v[b][j | z] : other;
                    }
              }
            } else {   // the parts, in order
#pragma unroll
              for (int j = 0; j < 4; ++j) v[0][j] = v[1][j] = 0.0f;
#pragma unroll 4
              for (int o = 0; o < parts; ++o) {
                const float* src = part_of(o) + min(c0 + (lane & 3), n - 1) * 128 + quarter * 32 + (lane & ~3);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                  const float4 x = __ldcg(reinterpret_cast<const float4*>(src + b * n * 128));
                  v[b][0] += x.x;
                  v[b][1] += x.y;
                  v[b][2] += x.z;
                  v[b][3] += x.w;
                }
              }
            }
            const int c = c0 + (lane & 3);
            const bool live = c < n;
            const int64_t hr = row0 + min(c, n - 1);
            const float gate = __shfl_sync(0xFFFFFFFFu, gates, c & 31);
            float h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)   // __fdividef: 2 ulp of 32 bits, far below what the pieces of h keep
              h[j] = gate * __fdividef(v[0][j], 1.0f + expf(-v[0][j])) * v[1][j];
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) m = max(m, __float_as_uint(h[j]) & 0x7FFFFFFFu);
#pragma unroll
            for (int z = 4; z < (FMT == DEC_NV ? 16 : 32); z *= 2) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, z));
            const int eb = block_exponent(m);
            if (live && (lane & (FMT == DEC_NV ? 12 : 28)) == 0)
              p.h.exps[hr * p.h_steps * EB + (FMT == DEC_NV ? k0 >> 4 : k0 >> 5)] = static_cast<uint8_t>(eb + 127);
            if constexpr (FMT == DEC_NV) {
              const int lo = m == 0u ? 128 : eb;
              const int t = max(eb, __shfl_xor_sync(0xFFFFFFFFu, eb, 16));
              const int l = min(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, 16));
              if (live && (lane & 28) == 0) {
                atomicMax(p.h.top + hr, t);
                atomicMin(p.h.low + hr, l);
              }
            }
            const uint64_t inv2 = f2_pack(block_multiplier<FMT>(eb), block_multiplier<FMT>(eb));
            uint64_t ra = f2_mul(f2_pack(h[0], h[1]), inv2), rb = f2_mul(f2_pack(h[2], h[3]), inv2);
            uint8_t* dst = p.h.codes + hr * PH * pitch + (FMT == DEC_NV ? k0 >> 1 : k0);
#pragma unroll
            for (int d = 0; d < PH; ++d, dst += pitch) {
              const uint64_t a = d + 1 < PH ? next_piece<FMT, false>(ra) : next_piece<FMT, true>(ra);
              const uint64_t b = d + 1 < PH ? next_piece<FMT, false>(rb) : next_piece<FMT, true>(rb);
              if (!live) continue;
              if constexpr (FMT == DEC_NV) *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(e2m1x4_f2(a, b));
              else *reinterpret_cast<uint32_t*>(dst) = e4m3x2_f2(a) | (e4m3x2_f2(b) << 16);
            }
          }
          if (phase == 0 || !share) release();
        }
      }
      i += i < n_share ? n_share : su;
      q.f = p.steps - 1;   // on from the last step of what was done
      q.acc = ACCS - 1;
      advance(q, i - 1);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L.tmem_cols);
  }
}

// h of the pairs (NVFP4, `blocks` blocks a row), between UP and DOWN: the row's largest exponent is known only now.
// Blocks more than NV_SPAN binades below it are written again under the smallest scale, as k_split_x does with x:
// the five digits as one integer, divided by the power of two between the scales, rounded to nearest.  Seldom needed
// (a row with values 2^17 apart), and only such a row is read.
// The launch costs a call 0 to 1.4 us: one token on 64 experts 2048x1408 19.3 -> 20.3, 64 tokens 68.3 -> 69.8, 8 experts
// 4096x14336 142.9 -> 144.7.  Left to UP's last warp per expert, which needs a fence and a count after every unit: 20.4,
// 76.0 and 149.2 us.
__global__ void __launch_bounds__(LIFT_THREADS) k_lift_low_blocks(const DecOperand h, int steps, int blocks) {
  constexpr int P = dec_pieces(DEC_NV, DEC_DOWN);
  pdl_launch_dependents();
  pdl_wait();
  const int row = blockIdx.x;
  const int lowest = h.top[row] - NV_SPAN;
  if (h.low[row] >= lowest) return;
  const int64_t pitch = static_cast<int64_t>(steps) * 128;
  uint8_t* exps = h.exps + static_cast<int64_t>(row) * steps * dec_exp_bytes(DEC_NV);
  uint8_t* codes = h.codes + static_cast<int64_t>(row) * P * pitch;
  for (int b = threadIdx.x; b < blocks; b += LIFT_THREADS) {
    const int shift = lowest + 127 - static_cast<int>(exps[b]);
    if (shift <= 0) continue;
    uint2 in[P], out[P];
#pragma unroll
    for (int d = 0; d < P; ++d) {
      in[d] = *reinterpret_cast<const uint2*>(codes + d * pitch + b * 8);
      out[d] = make_uint2(0u, 0u);
    }
#pragma unroll 1
    for (int z = 0; z < 64; z += 4) {   // one value: bits z % 32 of either word
      const bool hi = z >= 32;
      const int at = z & 31;
      int v = 0;
#pragma unroll
      for (int d = 0; d < P; ++d) {
        const uint32_t c = ((hi ? in[d].y : in[d].x) >> at) & 15u;
        const int m = (c & 7u) < 4u ? static_cast<int>(c & 7u) >> 1 : static_cast<int>(c & 7u) - 2;   // 0 1 2 3 4
        v = v * 8 + ((c & 8u) != 0u ? -m : m);
      }
      // |v| < 2^15: to nearest, halves away from zero
      const int a = shift > 16 ? 0 : (abs(v) + (1 << (shift - 1))) >> shift;
      v = v < 0 ? -a : a;
#pragma unroll
      for (int d = P - 1; d >= 0; --d) {
        const int digit = d == 0 ? v : ((v + 4) & 7) - 4;
        v = (v - digit) >> 3;
        const uint32_t m = static_cast<uint32_t>(abs(digit));
        const uint32_t c = (m < 3u ? m * 2u : m + 2u) | (digit < 0 ? 8u : 0u);
        if (hi) out[d].y |= c << at;
        else out[d].x |= c << at;
      }
    }
#pragma unroll
    for (int d = 0; d < P; ++d) *reinterpret_cast<uint2*>(codes + d * pitch + b * 8) = out[d];
    exps[b] = static_cast<uint8_t>(lowest + 127);
  }
}

// out[t] = sum of the pairs' rows y[row_of[t, j]], j in order (-1: none).  Four columns per thread.
__global__ void __launch_bounds__(256) k_sum_rows(const float* y, const int* row_of, int k, int H, uint16_t* out) {
  pdl_wait();
  const int t = blockIdx.x, c = (blockIdx.y * 256 + threadIdx.x) * 4;
  if (c >= H) return;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int j = 0; j < k; ++j) {
    const int r = row_of[t * k + j];
    if (r < 0) continue;
    const float4 x = *reinterpret_cast<const float4*>(y + static_cast<int64_t>(r) * H + c);
    v.x += x.x;
    v.y += x.y;
    v.z += x.z;
    v.w += x.w;
  }
  *reinterpret_cast<uint2*>(out + static_cast<int64_t>(t) * H + c) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// ---- host side -------------------------------------------------------------------------------

// 2-D byte matrix [rows, cols] (row pitch = cols) in boxes of box_rows rows x 128 bytes, 128-byte swizzle.
bool make_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {cols};
  const cuuint32_t box[2] = {128, box_rows}, estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int round_up(int v, int m) { return (v + m - 1) / m * m; }

// Shared memory for units of `rows` activation rows: half an SM where that holds three stages, else a whole one.
// MXFP8 experts with units for all CTAs take a whole one too (`many`): 64 experts 2048x1408, 64 tokens 101 us against
// 104, 8 experts 4096x14336, 64 tokens 231 against 235.  Elsewhere two CTAs are better, as said at the top.
bool dec_layout(int fmt, int mode, int rows, int E, int max_active, bool many, DecLayout* out) {
  const int n = round_up(dec_pieces(fmt, mode) * rows, 16);
  DecLayout L{};
  L.b_stage = n * 128;
  L.sfb_stage = dec_atoms(fmt) * ((n + 127) / 128) * 512;
  L.n_max = n;
  L.sf_cols = 4 * dec_atoms(fmt) * (1 + (n + 127) / 128);
  const int sfa = dec_atoms(fmt) * 512, bars = 384;
  const int fixed = 1024 + bars + (mode == DEC_LINEAR ? 0 : round_up(E * 8 + max_active * 12, 16));
  const int stage = DEC_A_STAGE + sfa + L.b_stage + L.sfb_stage;
  L.smem = DEC_SMEM_HALF;
  if ((L.smem - fixed) / stage < 3 || (fmt == DEC_MX && many)) L.smem = DEC_SMEM_FULL;
  L.stages = std::min(DEC_MAX_STAGES, (L.smem - fixed) / stage);
  L.tmem_cols = L.smem == DEC_SMEM_HALF ? DEC_TMEM_HALF : DEC_TMEM_FULL;
  // Two buffers of accumulators, where that leaves three sets of scales: the next unit's MMAs start while one is read
  // (NVFP4, 61x4096->28672: 21.7 us with, 25.1 without; fewer sets would hold up every step instead).
  for (L.acc_two = 1; L.acc_two >= 0; --L.acc_two) {
    L.sf_col = (mode == DEC_UP ? 2 : 1) * n << L.acc_two;
    L.sf_sets = std::min(L.stages, (static_cast<int>(L.tmem_cols) - L.sf_col) / L.sf_cols);
    if (L.sf_sets >= 3) break;
  }
  L.acc_two = std::max(L.acc_two, 0);
  if (L.stages < 3 || L.sf_sets < 2) return false;
  L.b = L.stages * DEC_A_STAGE;
  L.sfb = L.b + L.stages * L.b_stage;
  L.sfa = L.sfb + L.stages * L.sfb_stage;
  L.bars = L.sfa + L.stages * sfa;
  L.misc = L.bars + bars;
  *out = L;
  return true;
}
static_assert(2 * DEC_MAX_STAGES * 8 + 8 * 8 + 16 <= 384, "barriers and flags");
static_assert(dec_group(DEC_MX, DEC_DOWN) * 3 <= 160 && dec_group(DEC_MX, DEC_UP) * 2 * 2 <= 160 &&
                  dec_group(DEC_NV, DEC_UP) * 5 * 2 <= 160 && dec_group(DEC_NV, DEC_LINEAR) * 5 <= 160,
              "accumulators");

// Per-device set-up of one kernel instance (dynamic shared memory, and the carve-out that lets two CTAs
// share an SM); returns the number of SMs, 0 on failure.
template <int FMT, int MODE>
int dec_setup() {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> sms[kMaxDevices] = {};
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  if ((n = sms[dev].load()) > 0) return n;
  if (cudaFuncSetAttribute(k_decode<FMT, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, DEC_SMEM_FULL) !=
          cudaSuccess ||
      cudaFuncSetAttribute(k_decode<FMT, MODE>, cudaFuncAttributePreferredSharedMemoryCarveout,
                           cudaSharedmemCarveoutMaxShared) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  sms[dev].store(n);
  return n;
}

// Launch configuration: may start while the kernel before it in the stream ends (the kernels wait for
// that one themselves).
struct DecLaunch {
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg;
  DecLaunch(int grid, int threads, int smem, cudaStream_t stream) : cfg{} {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
};

template <int FMT, int MODE>
bool dec_launch(const CUtensorMap& tm_w, const CUtensorMap& tm_x, const DecParams& p, int sms, cudaStream_t stream) {
  const int ctas = p.L.smem == DEC_SMEM_HALF ? 2 * sms : sms;
  DecLaunch l(ctas / p.chunks * p.chunks, dec_threads(MODE), p.L.smem, stream);
  return cudaLaunchKernelEx(&l.cfg, k_decode<FMT, MODE>, tm_w, tm_x, p) == cudaSuccess;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
constexpr size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// Columns of `rows` rows of K values in `pieces` pieces each, from byte `at` of a workspace.
struct DecOperandLayout {
  size_t codes, exps, top, low, end;
  int64_t code_rows, steps;
  int pieces;
};
DecOperandLayout dec_operand(int fmt, int pieces, size_t at, int64_t rows, int64_t K) {
  DecOperandLayout o{};
  o.pieces = pieces;
  o.steps = (K + dec_step_values(fmt) - 1) / dec_step_values(fmt);
  o.code_rows = rows * pieces;
  o.codes = at;
  o.exps = align256(o.codes + static_cast<size_t>(o.code_rows) * o.steps * 128);
  o.top = align256(o.exps + static_cast<size_t>(rows) * o.steps * dec_exp_bytes(fmt));
  o.low = align256(o.top + static_cast<size_t>(rows) * sizeof(int));
  o.end = align256(o.low + static_cast<size_t>(rows) * sizeof(int));
  return o;
}
DecOperand dec_pointers(uint8_t* base, const DecOperandLayout& o) {
  return {base + o.codes, base + o.exps, reinterpret_cast<int*>(base + o.top), reinterpret_cast<int*>(base + o.low)};
}

// Workspace sizes do not depend on the device: room for the parts of at most this many CTAs.
constexpr int DEC_MAX_CTAS = 320;

// Workspace of the MoE layer: error word (256 bytes), columns of x and of h, rows of y, routing weights and
// numbers of the pairs, counters, parts.
struct DecWs {
  DecOperandLayout x, h;
  size_t y, gate, row_of, counters, part, end;
  int64_t n_up, n_down;   // counters of the two kernels
  int max_active;
};
bool dec_ws_layout(int fmt, int64_t T, int k, int64_t H, int64_t F, int E, DecWs* out) {
  if (T < 0 || T > DEC_MAX_TOKENS || k < 1 || k > DEC_MAX_K || E < 1 || E > 1024 || H <= 0 || F <= 0 ||
      H > INT32_MAX || F > INT32_MAX)
    return false;
  DecWs w{};
  const int64_t pairs = T * k;
  const int group = dec_group(fmt, DEC_UP);
  w.max_active = static_cast<int>(std::min<int64_t>(E, pairs) + (T > group ? pairs / group : 0));
  w.x = dec_operand(fmt, dec_pieces(fmt, DEC_UP), 256, pairs, H);
  w.h = dec_operand(fmt, dec_pieces(fmt, DEC_DOWN), w.x.end, pairs, F);
  // only units that are shared use counters, and those are fewer than the CTAs
  w.n_up = 4 * std::min<int64_t>(w.max_active * ((F + 127) / 128), DEC_MAX_CTAS);
  w.n_down = 4 * std::min<int64_t>(std::max<int64_t>(w.max_active, 1) * ((H + 127) / 128), DEC_MAX_CTAS);
  w.y = w.h.end;
  w.gate = align256(w.y + static_cast<size_t>(pairs) * H * sizeof(float));
  w.row_of = align256(w.gate + static_cast<size_t>(pairs) * sizeof(float));
  w.counters = align256(w.row_of + static_cast<size_t>(pairs) * sizeof(int));
  w.part = align256(w.counters + static_cast<size_t>(w.n_up + w.n_down) * sizeof(int));
  w.end = w.part + static_cast<size_t>(DEC_MAX_CTAS) * 2 * std::min<int64_t>(T, group) * 128 * sizeof(float);
  *out = w;
  return true;
}

// Workspace of a linear: error word, columns of x, counters, parts.
struct LinWs {
  DecOperandLayout x;
  size_t counters, part, end;
  int64_t n_counters;
};
LinWs lin_ws_layout(int fmt, int64_t T, int64_t K) {
  LinWs w{};
  w.x = dec_operand(fmt, dec_pieces(fmt, DEC_LINEAR), 256, T, K);
  w.n_counters = 4 * DEC_MAX_CTAS;   // chunks * units that are shared: fewer than the CTAs
  w.counters = w.x.end;
  w.part = align256(w.counters + static_cast<size_t>(w.n_counters) * sizeof(int));
  w.end = w.part + static_cast<size_t>(DEC_MAX_CTAS) * std::min<int64_t>(T, dec_group(fmt, DEC_LINEAR)) * 128 * sizeof(float);
  return w;
}

// The first kernel of a call (see k_split_x).
template <int FMT, bool BY_PAIR>
bool split_launch(const SplitParams& q, cudaStream_t stream) {
  DecLaunch l(BY_PAIR ? q.T * q.k : q.T, std::min(SPLIT_THREADS, round_up(q.K / (FMT == DEC_NV ? 16 : 8), 32)), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, k_split_x<FMT, BY_PAIR>, q) == cudaSuccess;
}

template <int FMT>
int moe_decode(const void* x, int64_t T, int64_t H, int64_t F, int E, int k, const int32_t* experts,
               const float* gates, const uint8_t* w1_q, const uint8_t* w1_sf, const float* w1_amax,
               const uint8_t* w2_q, const uint8_t* w2_sf, const float* w2_amax, void* out, void* workspace,
               size_t workspace_bytes, void* stream) {
  if (T < 0 || E < 1 || E > 1024 || k < 1 || H <= 0 || F <= 0) return MXFP8_ERR_INVALID_ARG;
  if (T > DEC_MAX_TOKENS || k > DEC_MAX_K || H % 128 != 0 || F % 128 != 0 || H > INT32_MAX || F > INT32_MAX)
    return MXFP8_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(E) * 2 * F > INT32_MAX || static_cast<int64_t>(E) * H > INT32_MAX)
    return MXFP8_ERR_UNSUPPORTED;
  DecWs ws;
  if (!dec_ws_layout(FMT, T, k, H, F, E, &ws)) return MXFP8_ERR_UNSUPPORTED;
  if (workspace == nullptr) return MXFP8_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < ws.end) return MXFP8_ERR_WORKSPACE;
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
  // steps of all units, as the kernels count them
  const int64_t act = ws.max_active;
  if (std::max<int64_t>(act * (F / 128), DEC_MAX_CTAS) * 2 * ws.x.steps > INT32_MAX ||
      std::max<int64_t>(act * (H / 128), DEC_MAX_CTAS) * ws.h.steps > INT32_MAX)
    return MXFP8_ERR_UNSUPPORTED;

  uint8_t* w = static_cast<uint8_t*>(workspace);
  const uint64_t per_byte = FMT == DEC_NV ? 2 : 1;   // values per code byte
  const int group = std::min(static_cast<int>(T), dec_group(FMT, DEC_UP));
  CUtensorMap m1, m2, mx, mh;
  if (!make_map(&m1, w1_q, static_cast<uint64_t>(E) * 2 * F, H / per_byte, 128) ||
      !make_map(&m2, w2_q, static_cast<uint64_t>(E) * H, F / per_byte, 128) ||
      !make_map(&mx, w + ws.x.codes, ws.x.code_rows, ws.x.steps * 128, ws.x.pieces * group) ||
      !make_map(&mh, w + ws.h.codes, ws.h.code_rows, ws.h.steps * 128, ws.h.pieces * group))
    return MXFP8_ERR_CUDA;
  const int sms = std::min(dec_setup<FMT, DEC_UP>(), dec_setup<FMT, DEC_DOWN>());
  if (sms <= 0 || 2 * sms > DEC_MAX_CTAS) return MXFP8_ERR_CUDA;

  DecParams up{};
  up.in = dec_pointers(w, ws.x);
  up.h = dec_pointers(w, ws.h);
  up.h_steps = static_cast<int>(ws.h.steps);
  up.experts = experts;
  up.gate = reinterpret_cast<float*>(w + ws.gate);
  up.y = reinterpret_cast<float*>(w + ws.y);
  up.err = reinterpret_cast<uint32_t*>(w);
  up.part = reinterpret_cast<float*>(w + ws.part);
  up.part_slot = 2 * group * 128;
  up.counters = reinterpret_cast<int*>(w + ws.counters);
  up.T = static_cast<int>(T);
  up.k = k;
  up.E = E;
  up.max_active = ws.max_active;
  up.chunks = 1;
  up.box_rows = group;
  up.timeout_ns = pipeline_wait_ns();
  up.drain_ns = kWaitTimeoutNs;
  DecParams down = up;
  up.w_sf = w1_sf;
  up.w_amax = w1_amax;
  up.K = static_cast<int>(H);
  up.steps = static_cast<int>(ws.x.steps);
  up.kt = up.steps * dec_atoms(FMT);
  up.tiles = static_cast<int>(F / 128);
  down.in = up.h;
  down.counters += ws.n_up;
  down.w_sf = w2_sf;
  down.w_amax = w2_amax;
  down.K = static_cast<int>(F);
  down.steps = up.h_steps;
  down.kt = down.steps * dec_atoms(FMT);
  down.tiles = static_cast<int>(H / 128);
  if (!dec_layout(FMT, DEC_UP, group, E, ws.max_active, act * up.tiles >= 2 * sms, &up.L) ||
      !dec_layout(FMT, DEC_DOWN, group, E, ws.max_active, act * down.tiles >= 2 * sms, &down.L))
    return MXFP8_ERR_UNSUPPORTED;

  SplitParams q{};
  q.x = static_cast<const uint16_t*>(x);
  q.o = up.in;
  q.err = up.err;
  q.experts = experts;
  q.gates = gates;
  q.gate = const_cast<float*>(up.gate);
  q.row_of = reinterpret_cast<int*>(w + ws.row_of);
  q.h_top = up.h.top;
  q.h_low = up.h.low;
  q.counters = up.counters;
  q.T = up.T;
  q.K = up.K;
  q.steps = up.steps;
  q.n_ids = up.T * k;
  q.E = E;
  q.k = k;
  q.n_top = FMT == DEC_NV ? up.T * k : 0;
  q.n_counters = static_cast<int>(ws.n_up + ws.n_down);
  if (!split_launch<FMT, true>(q, s) || !dec_launch<FMT, DEC_UP>(m1, mx, up, sms, s)) return MXFP8_ERR_CUDA;
  if constexpr (FMT == DEC_NV) {
    DecLaunch lift(up.T * k, LIFT_THREADS, 0, s);
    if (cudaLaunchKernelEx(&lift.cfg, k_lift_low_blocks, up.h, up.h_steps, down.K / 16) != cudaSuccess)
      return MXFP8_ERR_CUDA;
  }
  if (!dec_launch<FMT, DEC_DOWN>(m2, mh, down, sms, s)) return MXFP8_ERR_CUDA;
  DecLaunch sum(up.T, 256, 0, s);
  sum.cfg.gridDim.y = static_cast<unsigned>((H / 4 + 255) / 256);
  return cudaLaunchKernelEx(&sum.cfg, k_sum_rows, static_cast<const float*>(down.y), static_cast<const int*>(q.row_of), k,
                            static_cast<int>(H), static_cast<uint16_t*>(out)) == cudaSuccess
             ? MXFP8_OK
             : MXFP8_ERR_CUDA;
}

template <int FMT>
int matvec(const void* x, int64_t T, int64_t K, int64_t N, const uint8_t* w_q, const uint8_t* w_sf,
           const float* w_amax, void* y, void* workspace, size_t workspace_bytes, void* stream) {
  if (T < 0 || K <= 0 || N < 0) return MXFP8_ERR_INVALID_ARG;
  if (T > DEC_MAX_TOKENS || K % 128 != 0 || N % 128 != 0 || K > INT32_MAX || N > INT32_MAX) return MXFP8_ERR_UNSUPPORTED;
  const LinWs ws = lin_ws_layout(FMT, T, K);
  if (std::max<int64_t>(N / 128, DEC_MAX_CTAS) * ws.x.steps > INT32_MAX) return MXFP8_ERR_UNSUPPORTED;
  if (workspace == nullptr) return MXFP8_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < ws.end) return MXFP8_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0 || N == 0)
    return cudaMemsetAsync(workspace, 0, sizeof(uint32_t), s) == cudaSuccess ? MXFP8_OK : MXFP8_ERR_CUDA;
  const void* ptrs[] = {x, w_q, w_sf, y};
  for (const void* q : ptrs)
    if (q == nullptr || !aligned16(q)) return MXFP8_ERR_INVALID_ARG;
  if (FMT == DEC_NV && w_amax == nullptr) return MXFP8_ERR_INVALID_ARG;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  DecParams p{};
  p.chunks = static_cast<int>((T + dec_group(FMT, DEC_LINEAR) - 1) / dec_group(FMT, DEC_LINEAR));
  p.per_chunk = static_cast<int>((T + p.chunks - 1) / p.chunks);
  p.box_rows = p.per_chunk;
  CUtensorMap m, mx;
  if (!make_map(&m, w_q, static_cast<uint64_t>(N), static_cast<uint64_t>(K) / (FMT == DEC_NV ? 2 : 1), 128) ||
      !make_map(&mx, w + ws.x.codes, ws.x.code_rows, ws.x.steps * 128, ws.x.pieces * p.box_rows))
    return MXFP8_ERR_CUDA;
  const int sms = dec_setup<FMT, DEC_LINEAR>();
  if (sms <= 0 || 2 * sms > DEC_MAX_CTAS) return MXFP8_ERR_CUDA;
  p.in = dec_pointers(w, ws.x);
  p.w_sf = w_sf;
  p.w_amax = w_amax;
  p.out = static_cast<uint16_t*>(y);
  p.err = reinterpret_cast<uint32_t*>(w);
  p.part = reinterpret_cast<float*>(w + ws.part);
  p.part_slot = p.per_chunk * 128;
  p.counters = reinterpret_cast<int*>(w + ws.counters);
  p.T = static_cast<int>(T);
  p.K = static_cast<int>(K);
  p.steps = static_cast<int>(ws.x.steps);
  p.kt = p.steps * dec_atoms(FMT);
  p.tiles = static_cast<int>(N / 128);
  p.timeout_ns = pipeline_wait_ns();
  p.drain_ns = kWaitTimeoutNs;
  if (!dec_layout(FMT, DEC_LINEAR, p.per_chunk, 0, 0, false, &p.L)) return MXFP8_ERR_UNSUPPORTED;
  SplitParams q{};
  q.x = static_cast<const uint16_t*>(x);
  q.o = p.in;
  q.err = p.err;
  q.counters = p.counters;
  q.n_counters = static_cast<int>(ws.n_counters);
  q.T = p.T;
  q.K = p.K;
  q.steps = p.steps;
  return split_launch<FMT, false>(q, s) && dec_launch<FMT, DEC_LINEAR>(m, mx, p, sms, s) ? MXFP8_OK : MXFP8_ERR_CUDA;
}

}  // namespace
}  // namespace mx

using namespace mx;

extern "C" {

size_t moe_decode_workspace_size(int64_t T, int k, int64_t H, int64_t F, int E) {
  DecWs mx, nv;   // enough for either weight format
  if (!dec_ws_layout(DEC_MX, T, k, H, F, E, &mx) || !dec_ws_layout(DEC_NV, T, k, H, F, E, &nv)) return 0;
  return std::max(mx.end, nv.end);
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

size_t matvec_workspace_size(int64_t T, int64_t K) {
  if (T < 0 || T > DEC_MAX_TOKENS || K <= 0 || K > INT32_MAX) return 0;
  return std::max(lin_ws_layout(DEC_MX, T, K).end, lin_ws_layout(DEC_NV, T, K).end);
}

int mxfp8_matvec(const void* x, int64_t T, int64_t K, int64_t N, const uint8_t* w_q, const uint8_t* w_sf, void* y,
                 void* workspace, size_t workspace_bytes, void* stream) {
  return matvec<DEC_MX>(x, T, K, N, w_q, w_sf, nullptr, y, workspace, workspace_bytes, stream);
}

int nvfp4_matvec(const void* x, int64_t T, int64_t K, int64_t N, const uint8_t* w_q, const uint8_t* w_sf,
                 const float* w_amax, void* y, void* workspace, size_t workspace_bytes, void* stream) {
  return matvec<DEC_NV>(x, T, K, N, w_q, w_sf, w_amax, y, workspace, workspace_bytes, stream);
}

}  // extern "C"

// cross_entropy.cu -- softmax cross entropy of a linear layer over a large vocabulary, and its gradient, without the
// logits in memory.
//
// For a row x_t with target y_t and the vocabulary's rows w_v (all bf16), z_tv = x_t . w_v in 32 bits:
//   lse_t = log sum_v exp(z_tv),  loss_t = lse_t - z_{t, y_t}
// and for gradients dloss_t and dlse_t:
//   dz_tv = (dloss_t + dlse_t) exp(z_tv - lse_t) - dloss_t [v = y_t]
//   dx_t = sum_v dz_tv w_v,   dw_v = sum_t dz_tv x_t
// A row with a negative target takes no part: loss 0, no gradient, whatever its x holds.
//
// What bounds it: the tensor cores (forward 2 T H V operations, backward 6 T H V: the logits again, then the two
// products), and for few rows the bytes of w.  One GEMM kernel, k_ce_gemm, does all four products on tcgen05 with
// bf16 operands and fp32 accumulators in TMEM; its modes differ in the operands' layout and in the epilogue:
//   CE_LSE  x w^T      -> per row and column tile: the largest logit and the sum of exponentials; the target's logit
//   CE_DZ   x w^T      -> dz of one piece of the vocabulary, bf16, in the workspace
//   CE_DW   dz^T x     -> dw of the piece            (both operands contract over their rows: M- and N-major tiles)
//   CE_DX   dz w       -> dx, in fp32 parts where the vocabulary has several pieces or is split over CTAs
// The forward computes every row, since lse is written for all.  The backward first packs the rows that take part, so that
// padding costs its products nothing and nothing it holds can reach dw (0 * NaN); for fewer rows dz's kernel writes zeros
// for the others instead, to dz and to a copy of x (rows as they are).  dz is rounded to bf16 (by at most 2^-8 of its value): it is the operand of two products
// whose results are rounded to bf16 as well.  It lives for one piece of the vocabulary only, at most half of a large one.
// Few rows have a kernel of their own, k_ce_few, which is bound by the bytes of w: CE_LSE up to CE_FEW_FWD rows, CE_DZ and
// CE_DX up to CE_FEW.  dw is k_ce_gemm's for any number of rows.
//
// Measured (GB300; rows x H x vocabulary):
//   forward   8192 x 4096 x 32000   1.03-1.21 ms = 1.78-2.09 PFLOP/s (cool and under sustained power; cuBLAS in bf16 1.72-1.88)
//             1 x 4096 x 32000      47 us = 5.6 TB/s
//   backward  8192 x 4096 x 32000   3.31-3.86 ms = 1.67-1.95 PFLOP/s (6 T H V operations)
//             1531 x 2048 x 50257, 30% padding: 461 us = 1.44 PFLOP/s (1072 rows fill five tiles of 256; two pieces)
//             5 x 1024 x 32000      42 us; reads w twice and writes dw, 197 MB: 4.7 TB/s
// The tensor pipe is active 85-88% of the time in the logits' and dw's products and 76% in dx's (2048 x 4096 x 16384, 512 and
// 128 tiles for 76 pairs).  Loops of one lane instead of whole warps around the copies and the products left it at 78%: a
// step's 512 cycles of products took the issuing lane nearly as long.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "launch_host.h"
#include "mx_device.cuh"
#include "mx_internal.h"
#include "mxfp8moe.h"

namespace mx {
namespace {

constexpr int CE_BK = 64;                          // K per stage: 64 bf16 = one 128-byte swizzle row
constexpr int CE_HALF = 128;                       // rows of A and of B that a CTA stages
constexpr int CE_STAGES = 6;
constexpr int CE_OP_BYTES = CE_HALF * CE_BK * 2;   // 16 KB per operand
constexpr int CE_STAGE_BYTES = 2 * CE_OP_BYTES;
constexpr int CE_THREADS = 384;
constexpr int CE_WARP_PRODUCER = 0;
constexpr int CE_WARP_MMA = 1;
constexpr int CE_EPI_WARP0 = 4;
constexpr int CE_EPI_WARPS = 8;
constexpr uint32_t CE_BAR_EPI = 1;                 // hardware barrier of the epilogue warps
constexpr int CE_BUF_BYTES = 2048;                 // a warp's staging tile: 32 rows x 32 bf16; two per warp
constexpr int CE_EPI_BYTES = CE_EPI_WARPS * 2 * CE_BUF_BYTES;
constexpr int ce_smem_bytes(int stages) {
  return stages * CE_STAGE_BYTES + CE_EPI_BYTES + (2 * stages + 5) * 8 + 16 + 1024;
}
constexpr int CE_SHORT = 2;                        // stages where K is few steps (dw of few rows): two CTAs per SM
static_assert(ce_smem_bytes(CE_STAGES) <= 232448 && ce_smem_bytes(CE_SHORT) <= 115712, "shared memory budget");
constexpr int CE_CHUNK = 16;                       // logits: K steps that the tensor core sums before fp32 adds take over
constexpr uint32_t CE_REGS_LOW = 56, CE_REGS_HIGH = 224;   // logits: warps 0-3, epilogue warps
static_assert(128 * CE_REGS_LOW + 256 * CE_REGS_HIGH == CE_THREADS * 168, "register split must equal the launch pool");
// Most elements of dz at a time, in bf16: half of the logits', at least CE_DZ_LEAST (64 MB, below which it is not worth
// another piece) and at most CE_DZ_MOST (256 MB; up to CE_FEW rows, whose dz is small beside w, CE_DZ_FEW).  With all of dz
// in one piece the workspace was larger than the logits.
constexpr int64_t CE_DZ_LEAST = int64_t(1) << 25, CE_DZ_MOST = int64_t(1) << 27, CE_DZ_FEW = int64_t(1) << 28;
// Most elements of dx's fp32 parts: an eighth of the logits' (a quarter of their bytes in bf16), within these; where the
// vocabulary has several pieces, dx once at the least.
constexpr int64_t CE_PARTS_LEAST = int64_t(1) << 23, CE_PARTS_MOST = int64_t(1) << 24;
constexpr int64_t CE_MIN_PIECE = 2048;             // vocabulary entries of a piece, whatever the rows
constexpr float LOG2E = 1.4426950408889634f;

enum { CE_LSE = 0, CE_DZ = 1, CE_DW = 2, CE_DX = 3 };

struct CeMeta {
  uint32_t error;
  int32_t n;          // rows that take part (backward)
  int32_t splits;     // shares of the vocabulary in dx
  float gain;         // dz is held divided by it
  int32_t reserved[60];
};
static_assert(sizeof(CeMeta) == 256, "header");

struct CeParams {
  CeMeta* meta;
  const int32_t* row_map;      // backward: row of packed row i
  int rows;                    // forward, and backward with rows as they are: T; otherwise 0: meta->n packed rows
  int V, v0, vcols;            // vocabulary; first entry and entries of this piece
  int H;
  int group_m;                 // row tiles that share a column tile before the next one is taken
  int splits;                  // rows as they are, CE_DX: shares of the piece; otherwise meta->splits
  int piece_steps;             // CE_DX: K steps of a whole piece, dealt out to the shares
  const void* targets;
  int wide_targets;
  const float* lse;
  const float* dloss;
  const float* dlse;
  float2* part;                // CE_LSE: [2 * column tiles][pitch] (largest logit, sum of exponentials relative to it)
  float* zy;                   // CE_LSE: the target's logit
  int64_t pitch;
  float* acc;                  // CE_DX: [splits][rows][H] fp32, or NULL: dx is written directly
  int last;                    // the vocabulary's last piece (where it is one share, dx is written with it)
  float* acc_w;                // CE_DW: [dw_splits][vcols][H] fp32, or NULL: dw is written directly
  int dw_splits;
  int dw_rows;                 // rows as they are, CE_DW: rows of dz (few rows: of both its pieces)
  int acc_add;
  uint16_t* dz;                // few rows, CE_DZ: [NT][dz_pitch]
  int64_t dz_pitch;
  int d_rows, d_cols;          // CE_DZ, CE_DW: extent of the map that is stored to
  uint16_t* dx;
  const uint4* x;              // rows as they are, CE_DZ of the first piece: x, and a copy with zeros for rows that take no
  uint4* xp;                   // part ([t_pad], few rows: twice)
  int t_pad;
  uint32_t* status;            // a call's first kernel: an error word per CTA; otherwise NULL, meta->error
  const uint32_t* join;        // the kernel after it: those words, to be added to meta->error
  int joins;
  uint64_t timeout_ns;
};

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// exp(v - top): the difference first, so that the largest logit's own term is 1 exactly, whatever its size.
__device__ __forceinline__ float exp_below(float v, float top) { return ex2((v - top) * LOG2E); }
__device__ __forceinline__ void ce_report(const CeParams& p, uint32_t bits) {
  atomicOr(p.status != nullptr ? p.status + blockIdx.x : &p.meta->error, bits);
}
// Programmatic dependent launches: every kernel of a call lets the next one start its set-up at once, and waits for
// the one before it (and so for all of them) before it touches what that one reads or writes.  dw needs nothing of dx,
// the kernel before it, and runs beside its end: dx lets it start once dz is complete, and dw waits for dx when it is done.
__device__ __forceinline__ void ce_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void ce_wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void ce_join(const CeParams& p, int thread, int threads) {
  uint32_t bits = 0;
  for (int i = thread; i < p.joins; i += threads) bits |= p.join[i];
  if (bits != 0) atomicOr(&p.meta->error, bits);
}
// dz is held divided by the largest |dloss| (of the finite ones of rows that take part; by the largest |dlse| where that is
// 2^64 times as large): where all rows weigh the same, the target's entry is then p - 1, which bf16 holds exactly for p
// near 0, and not the same weight rounded in every row (by up to 2^-8 and always the same way: 1 / n for a mean).
struct CeGain {
  uint32_t loss, lse;   // bits of the largest magnitudes
  __device__ __forceinline__ CeGain() : loss(0), lse(0) {}
  static __device__ __forceinline__ uint32_t bits(float v) {
    const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
    return b < 0x7F800000u ? b : 0u;
  }
  __device__ __forceinline__ void add(const CeParams& p, int64_t row) {
    loss = max(loss, bits(__ldg(p.dloss + row)));
    if (p.dlse != nullptr) lse = max(lse, bits(__ldg(p.dlse + row)));
  }
  __device__ __forceinline__ void join_warp() {
    loss = __reduce_max_sync(0xFFFFFFFFu, loss);
    lse = __reduce_max_sync(0xFFFFFFFFu, lse);
  }
  __device__ __forceinline__ float value() const {
    const bool small = (lse >> 23) > (loss >> 23) + 64;
    return loss != 0 && !small ? __uint_as_float(loss) : lse != 0 ? __uint_as_float(lse) : 1.0f;
  }
};
__device__ __forceinline__ int ce_rows(const CeParams& p) { return p.rows > 0 ? p.rows : p.meta->n; }
__device__ __forceinline__ int ce_shares(const CeParams& p) { return p.rows > 0 ? p.splits : p.meta->splits; }
__device__ __forceinline__ int64_t ce_target(const CeParams& p, int64_t row) {
  return p.wide_targets ? __ldg(static_cast<const long long*>(p.targets) + row)
                        : static_cast<int64_t>(__ldg(static_cast<const int32_t*>(p.targets) + row));
}
__device__ __forceinline__ bool ce_takes_part(const CeParams& p, int64_t row) {
  const int64_t y = ce_target(p, row);
  return y >= 0 && y < p.V;
}
// Rows as they are: the gain of this warp's rows i, i + n, ...; the first CTA reports targets that are too large.
__device__ __forceinline__ CeGain ce_find_gain(const CeParams& p, int i, int n) {
  CeGain g;
  bool bad = false;
  for (int t = i; t < p.rows; t += n) {
    const int64_t y = ce_target(p, t);
    if (y >= 0 && y < p.V) g.add(p, t);
    bad |= y >= p.V;
  }
  if (bad && blockIdx.x == 0) ce_report(p, ERR_TARGET_RANGE);
  g.join_warp();
  return g;
}

// Instruction descriptor of kind::f16: fp32 accumulator, bf16 A and B, K-major unless the M / N major bits are set.
__host__ __device__ constexpr uint32_t ce_idesc(uint32_t M, uint32_t N, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | ((N >> 3) << 17) |
         ((M >> 4) << 24);
}
// Shared memory descriptors in 128-byte swizzle, lower word (address, leading byte offset) and upper word (stride byte
// offset 1024, version 1, swizzle): K-major, rows of 128 bytes; or M- / N-major, boxes of 64 elements x 64 rows of K, 8 KB
// apart (leading byte offset).  A step of 16 along K is 32 bytes of every row, or 16 rows of 128 bytes.
template <bool MN>
__device__ __forceinline__ uint32_t ce_desc_lo(uint32_t saddr) {
  return ((saddr & 0x3FFFFu) >> 4) | ((MN ? 8192u >> 4 : 1u) << 16);
}
constexpr uint32_t CE_DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
template <bool MN>
constexpr uint32_t CE_DESC_K16 = (MN ? 2048u : 32u) >> 4;
template <int CG, bool ALWAYS>
__device__ __forceinline__ void ce_mma(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem), "r"(a_lo), "r"(b_lo), "r"(idesc),
        "r"(ALWAYS ? 1u : accumulate), "r"(CE_DESC_HI)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem), "r"(a_lo), "r"(b_lo), "r"(idesc),
        "r"(ALWAYS ? 1u : accumulate), "r"(CE_DESC_HI)
        : "memory");
}
// The products of one stage (K = 64); the first one overwrites the accumulator where `first`.
template <int CG, bool A_MN, bool B_MN>
__device__ __forceinline__ void ce_mma_stage(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool first) {
  ce_mma<CG, false>(d_tmem, a_lo, b_lo, idesc, first ? 0u : 1u);
#pragma unroll
  for (int k = 1; k < CE_BK / 16; ++k)
    ce_mma<CG, true>(d_tmem, a_lo + k * CE_DESC_K16<A_MN>, b_lo + k * CE_DESC_K16<B_MN>, idesc, 1u);
}
// One lane of a converged warp, always the same.
__device__ __forceinline__ bool ce_elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

template <uint32_t N>
__device__ __forceinline__ void ce_regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <uint32_t N>
__device__ __forceinline__ void ce_regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// 16 or 32 consecutive TMEM columns of this warp's 32 lanes.
__device__ __forceinline__ void ce_tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

template <int MODE>
__device__ __forceinline__ void ce_start() {
  if (MODE == CE_DX) ce_wait_before();
  ce_dependents();
  if (MODE == CE_DZ) ce_wait_before();
}

template <int N>
__device__ __forceinline__ void ce_tmem_ld(uint32_t taddr, uint32_t* r) {
  if constexpr (N == 16) ce_tmem_ld16(taddr, r);
  else tmem_ld_32x32b_x32(taddr, r);
}

struct CeUnits {
  int nm, nn, steps;           // row tiles, column tiles, K steps in all
  int split_steps;             // CE_DX, CE_DW: K steps of a share
  int total;
};
template <int MODE, int CG>
__device__ __forceinline__ CeUnits ce_units(const CeParams& p) {
  constexpr int TILE = CE_HALF * CG;
  auto up = [](int a, int b) { return (a + b - 1) / b; };
  CeUnits c;
  int splits = 1;
  if (MODE == CE_LSE) {
    c.nm = up(p.rows, TILE);
    c.nn = up(p.V, TILE);
    c.steps = up(p.H, CE_BK);
  } else if (MODE == CE_DZ) {
    c.nm = up(ce_rows(p), TILE);
    c.nn = up(p.vcols, TILE);
    c.steps = up(p.H, CE_BK);
  } else if (MODE == CE_DW) {
    c.nm = up(p.vcols, TILE);
    c.nn = up(p.H, TILE);
    c.steps = up(p.rows > 0 ? p.dw_rows : p.meta->n, CE_BK);
  } else {
    c.nm = up(ce_rows(p), TILE);
    c.nn = up(p.H, TILE);
    c.steps = up(p.vcols, CE_BK);
  }
  c.split_steps = c.steps;
  if (MODE == CE_DX) {
    c.split_steps = up(p.piece_steps, ce_shares(p));
    splits = up(c.steps, c.split_steps);
  }
  if (MODE == CE_DW && p.dw_splits > 1) {           // every share writes its part, one without rows zeros
    c.split_steps = max(1, up(c.steps, p.dw_splits));
    splits = p.dw_splits;
  }
  c.total = c.nm * c.nn * splits;
  return c;
}
struct CeTile {
  int m, n, split, k0, steps;  // row tile, column tile, share, first K step and their number
};
// Unit u: shares outermost, then groups of group_m row tiles, in each the row tiles of one column tile after another.
template <int MODE>
__device__ __forceinline__ CeTile ce_tile(int u, const CeUnits& c, const CeParams& p) {
  CeTile t;
  const int per = c.nm * c.nn;
  constexpr bool SPLIT = MODE == CE_DX || MODE == CE_DW;
  t.split = SPLIT ? u / per : 0;
  const int w0 = u - t.split * per;
  const int g = w0 / (p.group_m * c.nn);
  const int in_g = min(p.group_m, c.nm - g * p.group_m);
  const int w = w0 - g * p.group_m * c.nn;
  t.n = w / in_g;
  t.m = g * p.group_m + (w - t.n * in_g);
  t.k0 = SPLIT ? t.split * c.split_steps : 0;
  t.steps = SPLIT ? max(0, min(c.split_steps, c.steps - t.k0)) : c.steps;
  return t;
}

// A phase that is complete already, without the cost of a wait.
__device__ __forceinline__ bool ce_ready(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait of one thread; a wait that runs out is reported and raises the abort flag of this CTA (and of its peer).
template <int CG>
__device__ __forceinline__ bool ce_wait(uint64_t* bar, uint32_t parity, bool cluster_scope, volatile int* abort,
                                        uint32_t peer_abort, const CeParams& p, uint32_t err_bit) {
  if (!(CG == 2 && cluster_scope) && ce_ready(bar, parity)) return true;
  if (CG == 2 && cluster_scope ? mbar_wait_cluster_bounded(bar, parity, abort, p.timeout_ns)
                               : mbar_wait_bounded(bar, parity, abort, p.timeout_ns))
    return true;
  ce_report(p, err_bit);
  *abort = 1;
  if (CG == 2) st_remote_u32(peer_abort, 1u);
  return false;
}

// The same by a whole warp, which agrees on the outcome.
template <int CG>
__device__ __forceinline__ bool ce_wait_warp(uint64_t* bar, uint32_t parity, bool cluster_scope, volatile int* abort,
                                             uint32_t peer_abort, const CeParams& p, uint32_t err_bit) {
  return __all_sync(0xFFFFFFFFu, ce_wait<CG>(bar, parity, cluster_scope, abort, peer_abort, p, err_bit)) != 0;
}

// CG = 1: a CTA computes tiles of 128 x 128.  CG = 2: a CTA pair computes tiles of 256 x 256, each CTA with 128 rows
// of A and of B in its shared memory and 128 rows of the result in its TMEM.  Either way a stage is 32 KB per CTA and
// the accumulators are double-buffered, so that an epilogue runs beside the next tile's products.
template <int MODE, int CG, int STAGES>
__global__ void __launch_bounds__(CE_THREADS, STAGES == CE_SHORT ? 2 : 1)
    k_ce_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
              const __grid_constant__ CUtensorMap tmD, const CeParams p) {
  constexpr bool A_MN = MODE == CE_DW, B_MN = MODE == CE_DW || MODE == CE_DX;
  constexpr int TILE = CE_HALF * CG;
  constexpr int NH = TILE / 2;                      // columns of an epilogue warp
  constexpr uint32_t TMEM_COLS = 2 * TILE;
  constexpr bool LOGITS = MODE == CE_LSE || MODE == CE_DZ;
  constexpr int CHUNK = LOGITS ? CE_CHUNK : 1 << 30;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * CE_STAGE_BYTES + CE_EPI_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* acc_full = empty + STAGES;           // [2]
  uint64_t* acc_empty = acc_full + 2;               // [2]
  uint64_t* drained = acc_empty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  uint32_t* gain_bits = tmem_holder + 2;            // [2]

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_cta_rank() : 0u;
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], CG * CE_EPI_WARPS);
    }
    mbar_init(drained, 1);
    *abort_flag = 0;
    gain_bits[0] = gain_bits[1] = 0u;
    if (p.status != nullptr) {                      // (the call's first kernel: nothing else writes these yet)
      p.status[blockIdx.x] = 0u;
      if (blockIdx.x == 0) p.meta->error = 0u;
    }
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == CE_WARP_MMA) {
    if constexpr (CG == 2) {
      tmem_alloc_pair(tmem_holder, TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_holder, TMEM_COLS);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();                  // the peer's barriers exist before anything arrives on them
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  ce_start<MODE>();
  const CeUnits units = ce_units<MODE, CG>(p);
  const int first = CG == 2 ? static_cast<int>(cluster_index()) : static_cast<int>(blockIdx.x);
  const int stride = CG == 2 ? static_cast<int>(cluster_count()) : static_cast<int>(gridDim.x);
  const uint32_t peer_abort = CG == 2 ? map_to_cta(const_cast<int*>(abort_flag), rank ^ 1u) : 0u;
  uint32_t prod_issued = 0;

  if (warp < CE_EPI_WARP0) {
    if constexpr (LOGITS) ce_regs_dec<CE_REGS_LOW>();
    if (warp == CE_WARP_PRODUCER) {
      // ---------------- tile copies (every CTA its own) ----------------
      // The warp runs the loop together, so that addresses stay in uniform registers, and one lane issues.
      const uint32_t leader_full = CG == 2 ? map_to_cta(full, 0) : 0u;
      uint32_t issued_parity = 0;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int u = first; ok && u < units.total; u += stride) {
        const CeTile t = ce_tile<MODE>(u, units, p);
        const int a0 = t.m * TILE + CE_HALF * static_cast<int>(rank);
        const int b0 = t.n * TILE + CE_HALF * static_cast<int>(rank);
        for (int s = 0; s < t.steps; ++s) {
          ok = ce_wait_warp<CG>(&empty[stage], phase ^ 1u, false, abort_flag, peer_abort, p, ERR_TIMEOUT_PRODUCER);
          if (!ok) break;
          if (ce_elect()) {
            uint8_t* sA = smem + stage * CE_STAGE_BYTES;
            uint8_t* sB = sA + CE_OP_BYTES;
            const int k = (t.k0 + s) * CE_BK;
            auto load = [&](uint8_t* dst, const CUtensorMap* map, int x, int y) {
              if constexpr (CG == 2) tma_load_2d_pair(dst, map, leader_full + stage * 8, x, y);
              else tma_load_2d(dst, map, &full[stage], x, y);
            };
            if (A_MN) {
              load(sA, &tmA, a0, k);
              load(sA + CE_OP_BYTES / 2, &tmA, a0 + 64, k);
            } else {
              load(sA, &tmA, k, a0);
            }
            // B rows: the vocabulary from v0 (logits), or K rows of it (dx)
            if (B_MN) {
              const int ky = MODE == CE_DX ? p.v0 + k : k;
              load(sB, &tmB, b0, ky);
              load(sB + CE_OP_BYTES / 2, &tmB, b0 + 64, ky);
            } else {
              load(sB, &tmB, k, p.v0 + b0);
            }
            if (leader) mbar_arrive_expect_tx(&full[stage], CG * CE_STAGE_BYTES);
          }
          __syncwarp();
          prod_issued |= 1u << stage;
          issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // Copies land before the CTA exits: the leader waits for its stages (their barriers count both CTAs' copies);
      // the second CTA's wait for the leader is the pair's closing barriers below.
      // (After an abort the second CTA may never have copied its half: then one wait is enough for this CTA's.)
      if (leader && lane == 0)
        for (int s = 0; s < STAGES; ++s)
          if (((prod_issued >> s) & 1u) &&
              !mbar_wait_bounded(&full[s], (issued_parity >> s) & 1u, nullptr, kWaitTimeoutNs)) {
            ce_report(p, ERR_TIMEOUT_DRAIN);
            break;
          }
      __syncwarp();
    } else if (warp == CE_WARP_MMA && leader) {
      // ---------------- MMA issuer (leader) ----------------
      // The warp runs the loop together, so that addresses stay in uniform registers, and one lane issues.
      constexpr uint32_t idesc = ce_idesc(TILE, TILE, A_MN, B_MN);
      const uint32_t a_lo = ce_desc_lo<A_MN>(smem_u32(smem)), b_lo = ce_desc_lo<B_MN>(smem_u32(smem) + CE_OP_BYTES);
      int stage = 0, buf = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool issued = false, ok = true;
      for (int u = first; ok && u < units.total; u += stride) {
        const CeTile t = ce_tile<MODE>(u, units, p);
        if (t.steps == 0) continue;                 // no rows: the epilogue writes zeros without the accumulator
        for (int s = 0; s < t.steps; ++s) {
          const bool opens = s % CHUNK == 0, closes = (s + 1) % CHUNK == 0 || s + 1 == t.steps;
          if (opens) ok = ce_wait_warp<CG>(&acc_empty[buf], acc_phase ^ 1u, true, abort_flag, peer_abort, p, ERR_TIMEOUT_MMA);
          ok = ok && ce_wait_warp<CG>(&full[stage], phase, false, abort_flag, peer_abort, p, ERR_TIMEOUT_MMA);
          if (!ok) break;
          tc_fence_after();
          if (ce_elect()) {
            const uint32_t at = stage * (CE_STAGE_BYTES >> 4);
            ce_mma_stage<CG, A_MN, B_MN>(tmem + buf * TILE, a_lo + at, b_lo + at, idesc, opens);
            if constexpr (CG == 2) tc_commit_pair_both(&empty[stage]);
            else tc_commit(&empty[stage]);
            if (closes) {
              if constexpr (CG == 2) tc_commit_pair_both(&acc_full[buf]);
              else tc_commit(&acc_full[buf]);
            }
          }
          __syncwarp();
          issued = true;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
          if (closes) {
            buf ^= 1;
            if (buf == 0) acc_phase ^= 1u;
          }
        }
      }
      if (issued && ce_elect()) {
        if constexpr (CG == 2) tc_commit_pair_local(drained);
        else tc_commit(drained);
        if (!mbar_wait_bounded(drained, 0, nullptr, kWaitTimeoutNs)) ce_report(p, ERR_TIMEOUT_DRAIN);
      }
      __syncwarp();
    } else if (MODE == CE_DZ && warp >= 2 && p.xp != nullptr) {
      // ---------------- rows as they are: the copy of x for dw, with zeros for rows that take no part ----------------
      const uint32_t per_row = static_cast<uint32_t>(p.H) / 8, total = static_cast<uint32_t>(p.t_pad) * per_row;
#pragma unroll 8
      for (uint32_t e = blockIdx.x * 64 + (threadIdx.x - 64); e < total; e += gridDim.x * 64) {
        const uint32_t r = e / per_row;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (r < static_cast<uint32_t>(p.rows)) {
          v = __ldg(p.x + e);
          if (!ce_takes_part(p, r)) v = make_uint4(0u, 0u, 0u, 0u);
        }
        p.xp[e] = v;
      }
    }
  } else {
    if constexpr (LOGITS) ce_regs_inc<CE_REGS_HIGH>();
    // ---------------- epilogue (every CTA its 128 rows) ----------------
    const int quarter = warp & 3;
    const int half = (warp - CE_EPI_WARP0) >> 2;
    const uint32_t t_row = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + NH * half;
    uint8_t* wbuf = smem + STAGES * CE_STAGE_BYTES + (warp - CE_EPI_WARP0) * 2 * CE_BUF_BYTES;
    const int n_rows = MODE == CE_DW ? 0 : ce_rows(p);
    const bool as_is = MODE != CE_LSE && p.rows > 0;
    float gain = 1.0f;
    if (MODE == CE_DZ && as_is) {
      const int i = static_cast<int>(threadIdx.x) - 32 * CE_EPI_WARP0;
      CeGain g = ce_find_gain(p, i, CE_EPI_WARPS * 32);
      if (lane == 0) {
        atomicMax(gain_bits, g.loss);
        atomicMax(gain_bits + 1, g.lse);
      }
      __syncwarp();
      group_and(CE_BAR_EPI, CE_EPI_WARPS * 32, true);
      g.loss = *static_cast<volatile uint32_t*>(gain_bits);
      g.lse = *static_cast<volatile uint32_t*>(gain_bits + 1);
      gain = g.value();
      if (blockIdx.x == 0 && i == 0) p.meta->gain = gain;
    } else if (MODE != CE_LSE) {
      gain = p.meta->gain;
    }
    if (MODE == CE_DX && p.join != nullptr && blockIdx.x == 0)
      ce_join(p, static_cast<int>(threadIdx.x) - 32 * CE_EPI_WARP0, CE_EPI_WARPS * 32);
    const bool dx_direct = MODE == CE_DX && (p.acc == nullptr || (p.last && ce_shares(p) == 1));
    int buf = 0;
    uint32_t acc_phase = 0;
    for (int u = first; u < units.total; u += stride) {
      const CeTile t = ce_tile<MODE>(u, units, p);
      const int row0 = t.m * TILE + CE_HALF * static_cast<int>(rank) + quarter * 32;
      const int row = row0 + lane;
      const int col0 = t.n * TILE + NH * half;
      // what the row needs besides its logits, before the wait
      int y = -1;                                   // the target's column; outside every tile without one
      float rate = 0.0f, hot = 0.0f, lse = 0.0f;
      int src = 0;
      if (MODE == CE_LSE && row < n_rows) {
        const int64_t target = ce_target(p, row);
        y = target < p.V ? static_cast<int>(max(target, int64_t(-1))) : -1;
      }
      bool in = row < n_rows;                       // the row takes part
      if ((MODE == CE_DZ || MODE == CE_DX) && in) {
        src = as_is ? row : __ldg(p.row_map + row);
        if (as_is) in = ce_takes_part(p, row);
      }
      if (MODE == CE_DZ && in) {
        y = static_cast<int>(ce_target(p, src)) - p.v0;
        hot = __ldg(p.dloss + src) / gain;
        rate = hot + (p.dlse != nullptr ? __ldg(p.dlse + src) / gain : 0.0f);
        lse = __ldg(p.lse + src);
      }
      auto wait_acc = [&]() {
        bool got = true;
        if (warp == CE_EPI_WARP0 && lane == 0)
          got = ce_wait<CG>(&acc_full[buf], acc_phase, false, abort_flag, peer_abort, p, ERR_TIMEOUT_EPILOGUE);
        __syncwarp();                               // (the barrier counts whole warps, whichever lanes come first)
        got = group_and(CE_BAR_EPI, CE_EPI_WARPS * 32, got);
        tc_fence_after();
        return got;
      };
      auto release_acc = [&]() {                    // all of this warp's columns have been read
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 2) mbar_arrive_remote(map_to_cta(&acc_empty[buf], 0));
          else mbar_arrive(&acc_empty[buf]);
        }
      };
      auto next_acc = [&]() {
        buf ^= 1;
        if (buf == 0) acc_phase ^= 1u;
      };
      // 32 columns from `col` on, as bf16, through a staging tile to the map that is stored to.
      auto put_bf16 = [&](int c, const uint32_t* v) {
        uint8_t* out = wbuf + ((c >> 5) & 1) * CE_BUF_BYTES;
        if (lane == 0) bulk_wait_read_le1();        // the store that last used this buffer has read it
        __syncwarp();
        // row `lane`: four 16-byte chunks, 64B swizzle (chunk j of row i at j ^ ((i >> 1) & 3))
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint4 o;
          o.x = pack_bf16x2(__uint_as_float(v[8 * j + 0]), __uint_as_float(v[8 * j + 1]));
          o.y = pack_bf16x2(__uint_as_float(v[8 * j + 2]), __uint_as_float(v[8 * j + 3]));
          o.z = pack_bf16x2(__uint_as_float(v[8 * j + 4]), __uint_as_float(v[8 * j + 5]));
          o.w = pack_bf16x2(__uint_as_float(v[8 * j + 6]), __uint_as_float(v[8 * j + 7]));
          *reinterpret_cast<uint4*>(out + lane * 64 + 16 * (j ^ ((lane >> 1) & 3))) = o;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (row0 < p.d_rows && col0 + c < p.d_cols) tma_store_2d(&tmD, out, col0 + c, row0);   // clipped at the edges
          bulk_commit_group();
        }
      };
      if constexpr (LOGITS) {
        // The tensor core cuts its sums off instead of rounding them, always towards zero: H = 4096 in one sum left loss
        // off by 2.8e-6 of its norm, an fp32 product by 0.6e-6.  So it sums CE_CHUNK steps at a time, and these are added
        // here, rounded: 0.6e-6 with 16 steps (1269 us for 8192 x 4096 x 32000), 1.4e-6 with 32 (1256), 0.3e-6 with 8 (1293).
        // The backward's logits are the forward's, bit for bit, so that p is 1 and dz 0 where the target is certain.
        float z[NH];
        bool ok = true;
        for (int s = 0; ok && s < t.steps; s += CE_CHUNK) {
          ok = wait_acc();
          if (ok) {
#pragma unroll
            for (int c = 0; c < NH; c += 32) {
              uint32_t v[32];
              tmem_ld_32x32b_x32(t_row + buf * TILE + c, v);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) z[c + i] = s == 0 ? __uint_as_float(v[i]) : z[c + i] + __uint_as_float(v[i]);
            }
            release_acc();
            next_acc();
          }
        }
        if (!ok) break;
        if constexpr (MODE == CE_DZ) {
#pragma unroll
          for (int c = 0; c < NH; c += 32) {
            uint32_t v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int col = col0 + c + i;
              float d = rate * exp_below(z[c + i], lse);
              if (y == col) d -= hot;
              v[i] = in && col < p.vcols ? __float_as_uint(d) : 0u;
            }
            put_bf16(c, v);
          }
          continue;
        }
        if (y >= col0 && y < col0 + NH) {
          const int at = y - col0;
          float zy = 0.0f;
#pragma unroll
          for (int i = 0; i < NH; ++i)
            if (i == at) zy = z[i];
          p.zy[row] = zy;
        }
        if (col0 + NH > p.V) {
#pragma unroll
          for (int i = 0; i < NH; ++i)
            if (col0 + i >= p.V) z[i] = -INFINITY;
        }
        float top = z[0];
#pragma unroll
        for (int i = 1; i < NH; ++i) top = fmaxf(top, z[i]);
        const float base = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NH; ++i) sum += exp_below(z[i], base);
        if (row < n_rows) p.part[(2 * t.n + half) * p.pitch + row] = make_float2(top, sum);
        continue;
      }
      if (t.steps > 0 && !wait_acc()) break;
#pragma unroll 1
      for (int c = 0; c < NH; c += 32) {
        uint32_t v[32];
        if (t.steps > 0) {
          tmem_ld_32x32b_x32(t_row + buf * TILE + c, v);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0u;
        }
        if (c + 32 >= NH && t.steps > 0) release_acc();
        const int col = col0 + c;
        if constexpr (MODE == CE_DW) {
          if (p.acc_w != nullptr) {
            float* dst = p.acc_w + (static_cast<int64_t>(t.split) * p.vcols + row) * p.H + col;
            if (row < p.vcols)
#pragma unroll
              for (int j = 0; j < 32; j += 8)
                if (col + j < p.H)
                  st_global_32B(dst + j, make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]),
                                make_uint4(v[j + 4], v[j + 5], v[j + 6], v[j + 7]));
            continue;
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * gain);
          put_bf16(c, v);
        } else if (row < n_rows) {                  // CE_DX
          float* part = p.acc + (static_cast<int64_t>(t.split) * n_rows + row) * p.H + col;
          if (p.acc_add) {                          // the pieces before this one; all loads first
            float4 old[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (col + 4 * j < p.H) old[j] = *reinterpret_cast<const float4*>(part + 4 * j);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (col + 4 * j < p.H) {
                v[4 * j + 0] = __float_as_uint(__uint_as_float(v[4 * j + 0]) + old[j].x);
                v[4 * j + 1] = __float_as_uint(__uint_as_float(v[4 * j + 1]) + old[j].y);
                v[4 * j + 2] = __float_as_uint(__uint_as_float(v[4 * j + 2]) + old[j].z);
                v[4 * j + 3] = __float_as_uint(__uint_as_float(v[4 * j + 3]) + old[j].w);
              }
          }
          if (dx_direct) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = in ? __float_as_uint(__uint_as_float(v[i]) * gain) : 0u;
            uint16_t* dst = p.dx + static_cast<int64_t>(src) * p.H + col;
#pragma unroll
            for (int j = 0; j < 32; j += 8)
              if (col + j < p.H) {
                uint4 o;
                o.x = pack_bf16x2(__uint_as_float(v[j + 0]), __uint_as_float(v[j + 1]));
                o.y = pack_bf16x2(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]));
                o.z = pack_bf16x2(__uint_as_float(v[j + 4]), __uint_as_float(v[j + 5]));
                o.w = pack_bf16x2(__uint_as_float(v[j + 6]), __uint_as_float(v[j + 7]));
                *reinterpret_cast<uint4*>(dst + j) = o;
              }
          } else {
#pragma unroll
            for (int j = 0; j < 32; j += 8)
              if (col + j < p.H)
                st_global_32B(part + j, make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]),
                              make_uint4(v[j + 4], v[j + 5], v[j + 6], v[j + 7]));
          }
        }
      }
      if (t.steps > 0) next_acc();
    }
    if ((MODE == CE_DZ || MODE == CE_DW) && lane == 0) bulk_wait_all();   // stores complete before exit
  }

  if (MODE == CE_DW) ce_wait_before();
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) {
    cluster_sync_all();   // all pair MMAs are done and no remote arrive targets an exited CTA
    // After an abort the second CTA's copies may still be in flight towards the leader's barriers: they depend on
    // nothing but memory and get a fixed 200 us to land before either CTA exits.
    if (!leader && warp == CE_WARP_PRODUCER && lane == 0 && prod_issued != 0 && *abort_flag) {
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 200000ull) {
      }
    }
    cluster_sync_all();
  }
  if (warp == CE_WARP_MMA) {
    __syncwarp();
    tc_fence_after();
    if constexpr (CG == 2) tmem_dealloc_pair(tmem, TMEM_COLS);
    else tmem_dealloc(tmem, TMEM_COLS);
  }
}

// ---- few rows -------------------------------------------------------------------------------
// Up to CE_FEW rows: the weights are the M operand (128 rows of w, or 128 columns for dx), the rows the N operand
// (NT of them), so that nothing is spent on rows that are not there and a CTA's stages hold little but weights.  Bound:
// the bytes of w.  Two CTAs per SM keep twice the copies in flight.
//   CE_LSE  (up to 32 rows) z^T = w x^T: a thread has one vocabulary entry and all rows; it carries every row's running
//           maximum and sum over all its tiles, and lanes are joined once, at the end
//   CE_DZ   the same product and dz; rows that take no part are zeros in dz and in a copy of x for dw (no packing)
//   CE_DX   dx^T = w^T dz^T over a share of the vocabulary: fp32 parts
// The tensor cores have time to spare here, so dz is held in two bf16 pieces, the second of what the first one leaves (to
// 2^-16 of it): NT rows of first pieces and NT of second ones, in dx's product as 2 NT columns, in dw's as 2 NT rows of K
// beside two copies of x.
constexpr int CE_FEW = 64;                         // rows; in the forward CE_FEW_FWD: 64 rows' maxima and sums leave room for
constexpr int CE_FEW_FWD = 32;                     // one CTA per SM (64 x 4096 x 32000: 57 us, as 128 rows of k_ce_gemm 53)
constexpr int CE_FEW_BUFS = 4;                     // accumulators of NT columns (dx: 2 NT)
constexpr int CE_FEW_CHUNK = 4;                    // as CE_CHUNK: the epilogue has time (2 and 8 steps measure the same)
template <int MODE, int NT>
struct FewShape {
  static constexpr int EPI_WARPS = NT == 64 ? 8 : 4;        // 64 rows are two threads' work per entry
  static constexpr int COLS = NT / (EPI_WARPS / 4);
  static constexpr int PER_SM = NT == 64 ? 1 : 2;
  static constexpr int THREADS = 64 + 32 * EPI_WARPS;
  static constexpr int NB = MODE == CE_DX ? 2 * NT : NT;    // rows of the N operand
  static constexpr int B_BYTES = NB * CE_BK * 2;
  static constexpr int STAGE_BYTES = CE_OP_BYTES + B_BYTES;
  static constexpr int STAGES = MODE == CE_DX ? (NT == 64 ? 6 : NT == 32 ? 4 : 5) : (NT == 64 ? 9 : NT == 32 ? 5 : 6);
  static constexpr int PARAM_OFFSET = STAGES * STAGE_BYTES;             // [NT] float4 (CE_DZ), [EPI_WARPS][COLS] float2 (CE_LSE)
  static constexpr int BAR_OFFSET = PARAM_OFFSET + EPI_WARPS * COLS * 16;
  static constexpr int SMEM_BYTES = BAR_OFFSET + (2 * STAGES + 2 * CE_FEW_BUFS + 1) * 8 + 8 + 1024;
  static_assert(MODE == CE_DZ || MODE == CE_DX || (MODE == CE_LSE && NT <= CE_FEW_FWD), "forms of the few rows' kernel");
  static_assert(SMEM_BYTES <= (PER_SM == 2 ? 115712 : 232448), "shared memory budget");
  static_assert(PER_SM * CE_FEW_BUFS * NB <= 512, "TMEM budget");
};

template <int MODE, int NT>
__global__ void __launch_bounds__(FewShape<MODE, NT>::THREADS, FewShape<MODE, NT>::PER_SM)
    k_ce_few(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const CeParams p) {
  using S = FewShape<MODE, NT>;
  constexpr bool A_MN = MODE == CE_DX;
  // (33 to 64 rows: the forward's logits are k_ce_gemm's)
  constexpr int CHUNK = MODE == CE_DX ? 1 << 30 : NT == 64 ? CE_CHUNK : CE_FEW_CHUNK;
  constexpr int NO_TARGET = INT_MIN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::BAR_OFFSET);
  uint64_t* empty = full + S::STAGES;
  uint64_t* acc_full = empty + S::STAGES;
  uint64_t* acc_empty = acc_full + CE_FEW_BUFS;
  uint64_t* drained = acc_empty + CE_FEW_BUFS;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // units: 128 vocabulary entries each, or (share of the piece, 128 columns of dx)
  const int tiles = MODE == CE_DX ? (p.H + 127) / 128 : (p.vcols + 127) / 128;
  const int k_steps = MODE == CE_DX ? (p.vcols + CE_BK - 1) / CE_BK : (p.H + CE_BK - 1) / CE_BK;
  const int split_steps = MODE == CE_DX ? (p.piece_steps + p.splits - 1) / p.splits : k_steps;
  const int total = MODE == CE_DX ? tiles * ((k_steps + split_steps - 1) / split_steps) : tiles;
  auto k_begin = [&](int u) { return MODE == CE_DX ? u / tiles * split_steps : 0; };
  auto k_end = [&](int u) { return MODE == CE_DX ? min(k_steps, (u / tiles + 1) * split_steps) : k_steps; };

  // The copies of the first stages need nothing of the kernel before (row packing, dz) but for the rows' half: the weights
  // are on their way while that one ends and while this one sets itself up.
  const int k_first = k_begin(blockIdx.x);
  const int early = min(S::STAGES, k_end(blockIdx.x) - k_first);
  auto load_w = [&](int stage, int m0, int ks) {
    uint8_t* sA = smem + stage * S::STAGE_BYTES;
    mbar_arrive_expect_tx(&full[stage], S::STAGE_BYTES);
    if (A_MN) {
      tma_load_2d(sA, &tmA, &full[stage], m0, p.v0 + ks * CE_BK);
      tma_load_2d(sA + CE_OP_BYTES / 2, &tmA, &full[stage], m0 + 64, p.v0 + ks * CE_BK);
    } else {
      tma_load_2d(sA, &tmA, &full[stage], ks * CE_BK, p.v0 + m0);
    }
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < CE_FEW_BUFS; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], S::EPI_WARPS);
    }
    mbar_init(drained, 1);
    *abort_flag = 0;
    if (p.status != nullptr) {                      // (the call's first kernel: nothing else writes these yet)
      p.status[blockIdx.x] = 0u;
      if (blockIdx.x == 0) p.meta->error = 0u;
    }
    fence_barrier_init();
    fence_proxy_async_smem();
    for (int s = 0; s < early; ++s) load_w(s, (MODE == CE_DX ? blockIdx.x % tiles : blockIdx.x) * 128, k_first + s);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, CE_FEW_BUFS * S::NB);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  // (the copying thread waits later, see there)
  if (threadIdx.x != 0) ce_start<MODE>();
  if (warp == 0) {
    // ---------------- tile copies (as in k_ce_gemm) ----------------
    if (lane == 0) ce_start<MODE>();
    __syncwarp();
    uint32_t issued = 0, issued_parity = 0;
    int stage = 0, ahead = early;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
      const int m0 = (MODE == CE_DX ? u % tiles : u) * 128;
      const int k1 = k_end(u);
      for (int ks = k_begin(u); ks < k1; ++ks) {
        ok = ce_wait_warp<1>(&empty[stage], phase ^ 1u, false, abort_flag, 0u, p, ERR_TIMEOUT_PRODUCER);
        if (!ok) break;
        if (ce_elect()) {
          if (ahead <= 0) load_w(stage, m0, ks);
          tma_load_2d(smem + stage * S::STAGE_BYTES + CE_OP_BYTES, &tmB, &full[stage], ks * CE_BK, 0);
        }
        __syncwarp();
        --ahead;
        issued |= 1u << stage;
        issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == S::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (lane == 0) {
      for (; ahead > 0; --ahead) {                  // (after an abort) the early stages get their other half
        tma_load_2d(smem + (early - ahead) * S::STAGE_BYTES + CE_OP_BYTES, &tmB, &full[early - ahead], 0, 0);
        issued |= 1u << (early - ahead);
      }
      for (int s = 0; s < S::STAGES; ++s)           // copies land before the CTA exits
        if ((issued >> s) & 1u)
          if (!mbar_wait_bounded(&full[s], (issued_parity >> s) & 1u, nullptr, kWaitTimeoutNs))
            ce_report(p, ERR_TIMEOUT_DRAIN);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMA issuer (as in k_ce_gemm) ----------------
    constexpr uint32_t idesc = ce_idesc(128, S::NB, A_MN, false);
    const uint32_t a_lo = ce_desc_lo<A_MN>(smem_u32(smem)), b_lo = ce_desc_lo<false>(smem_u32(smem) + CE_OP_BYTES);
    int stage = 0, buf = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool issued = false, ok = true;
    for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
      const int steps = k_end(u) - k_begin(u);
      for (int s = 0; s < steps; ++s) {
        const bool opens = s % CHUNK == 0, closes = (s + 1) % CHUNK == 0 || s + 1 == steps;
        if (opens) ok = ce_wait_warp<1>(&acc_empty[buf], acc_phase ^ 1u, false, abort_flag, 0u, p, ERR_TIMEOUT_MMA);
        ok = ok && ce_wait_warp<1>(&full[stage], phase, false, abort_flag, 0u, p, ERR_TIMEOUT_MMA);
        if (!ok) break;
        tc_fence_after();
        if (ce_elect()) {
          const uint32_t at = stage * (S::STAGE_BYTES >> 4);
          ce_mma_stage<1, A_MN, false>(tmem + buf * S::NB, a_lo + at, b_lo + at, idesc, opens);
          tc_commit(&empty[stage]);
          if (closes) tc_commit(&acc_full[buf]);
        }
        __syncwarp();
        issued = true;
        if (++stage == S::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
        if (closes && ++buf == CE_FEW_BUFS) {
          buf = 0;
          acc_phase ^= 1u;
        }
      }
    }
    if (issued && ce_elect()) {
      tc_commit(drained);
      if (!mbar_wait_bounded(drained, 0, nullptr, kWaitTimeoutNs)) ce_report(p, ERR_TIMEOUT_DRAIN);
    }
    __syncwarp();
  } else {
    // ---------------- epilogue ----------------
    const int quarter = warp & 3;
    const int c0 = (warp - 2) / 4 * S::COLS;        // first row (column of the accumulator) of this warp
    const uint32_t t_row = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + c0;
    const int n_rows = p.rows;
    // CE_DZ: what each row needs; CE_LSE: its target
    float4* s_row = reinterpret_cast<float4*>(smem + S::PARAM_OFFSET);
    float gain = 1.0f;
    if (MODE == CE_DX) gain = p.meta->gain;
    if (MODE != CE_DX) {
      const int i = static_cast<int>(threadIdx.x) - 64;
      if (MODE == CE_DZ) {
        gain = ce_find_gain(p, lane, 32).value();
        if (blockIdx.x == 0 && i == 0) p.meta->gain = gain;
      }
      if (i < NT) {
        float4 r = make_float4(0.0f, 0.0f, 0.0f, __int_as_float(NO_TARGET));
        if (i < n_rows) {
          const int64_t target = ce_target(p, i);
          if (target >= 0 && target < p.V) {
            r.w = __int_as_float(static_cast<int>(target) - p.v0);
            if (MODE == CE_DZ) {
              r.z = __ldg(p.dloss + i) / gain;
              r.x = r.z + (p.dlse != nullptr ? __ldg(p.dlse + i) / gain : 0.0f);
              r.y = __ldg(p.lse + i);
            }
          }
        }
        s_row[i] = r;
      }
      __syncwarp();
      asm volatile("bar.sync %0, %1;" ::"r"(CE_BAR_EPI), "r"(S::EPI_WARPS * 32) : "memory");
      if (MODE == CE_DZ && p.xp != nullptr)
        for (int r = blockIdx.x; r < NT; r += gridDim.x) {
          const bool in = __float_as_int(s_row[r].w) != NO_TARGET;
          const int64_t per_row = p.H / 8;
          for (int64_t c = i; c < per_row; c += S::EPI_WARPS * 32) {
            const uint4 o = in ? __ldg(p.x + r * per_row + c) : make_uint4(0u, 0u, 0u, 0u);
            p.xp[r * per_row + c] = o;
            p.xp[(NT + r) * per_row + c] = o;
          }
        }
    } else if (p.join != nullptr && blockIdx.x == 0) {
      ce_join(p, static_cast<int>(threadIdx.x) - 64, S::EPI_WARPS * 32);
    }
    // CE_LSE: below every logit, and finite, so that a first logit replaces it without a case of its own
    float m[S::COLS], sum[S::COLS];
    if (MODE == CE_LSE) {
#pragma unroll
      for (int j = 0; j < S::COLS; ++j) {
        m[j] = -3e38f;
        sum[j] = 0.0f;
      }
    }
    int buf = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
      const int steps = k_end(u) - k_begin(u);
      float z[S::COLS];
      for (int s = 0; s < steps; s += CHUNK < steps ? CHUNK : steps) {
        int got = 1;
        if (lane == 0) got = ce_wait<1>(&acc_full[buf], acc_phase, false, abort_flag, 0u, p, ERR_TIMEOUT_EPILOGUE) ? 1 : 0;
        ok = __shfl_sync(0xFFFFFFFFu, got, 0) != 0;
        if (!ok) break;
        tc_fence_after();
        uint32_t v[S::COLS];
        ce_tmem_ld<S::COLS>(t_row + buf * S::NB, v);
        uint32_t lo[MODE == CE_DX ? S::COLS : 1];
        if constexpr (MODE == CE_DX) ce_tmem_ld<S::COLS>(t_row + buf * S::NB + NT, lo);
        tmem_ld_wait();
        if constexpr (MODE == CE_DX) {
#pragma unroll
          for (int j = 0; j < S::COLS; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(lo[j]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[buf]);
        if (++buf == CE_FEW_BUFS) {
          buf = 0;
          acc_phase ^= 1u;
        }
#pragma unroll
        for (int j = 0; j < S::COLS; ++j) z[j] = s == 0 ? __uint_as_float(v[j]) : z[j] + __uint_as_float(v[j]);
      }
      if (!ok) break;
      if constexpr (MODE == CE_LSE) {
        const int v = u * 128 + quarter * 32 + lane;
        if (v < p.V) {
#pragma unroll
          for (int j = 0; j < S::COLS; ++j) {
            if (j % 8 == 0 && c0 + j >= n_rows) break;
            if (__float_as_int(s_row[c0 + j].w) == v) p.zy[c0 + j] = z[j];
            const float d = z[j] - m[j];
            const float e = ex2(-fabsf(d) * LOG2E);
            sum[j] = d > 0.0f ? fmaf(sum[j], e, 1.0f) : sum[j] + e;
            m[j] = fmaxf(m[j], z[j]);
          }
        }
      } else if constexpr (MODE == CE_DZ) {
        const int v = u * 128 + quarter * 32 + lane;
        uint16_t* dst = p.dz + static_cast<int64_t>(c0) * p.dz_pitch + v;
#pragma unroll
        for (int j = 0; j < S::COLS; ++j) {
          const float4 r = s_row[c0 + j];
          float d = r.x * exp_below(z[j], r.y);
          if (__float_as_int(r.w) == v) d -= r.z;
          const bool in = __float_as_int(r.w) != NO_TARGET && v < p.vcols;
          const __nv_bfloat16 hi = __float2bfloat16_rn(d), lo = __float2bfloat16_rn(d - __bfloat162float(hi));
          dst[j * p.dz_pitch] = in ? __bfloat16_as_ushort(hi) : 0;
          dst[(NT + j) * p.dz_pitch] = in ? __bfloat16_as_ushort(lo) : 0;
        }
      } else {
        const int h = u % tiles * 128 + quarter * 32 + lane;
        if (p.acc == nullptr) {
          if (h < p.H)
#pragma unroll
            for (int j = 0; j < S::COLS; ++j)
              if (c0 + j < n_rows)
                p.dx[static_cast<int64_t>(c0 + j) * p.H + h] =
                    ce_takes_part(p, c0 + j) ? __bfloat16_as_ushort(__float2bfloat16_rn(z[j] * gain)) : 0;
          continue;
        }
        float* dst = p.acc + (static_cast<int64_t>(u / tiles) * n_rows + c0) * p.H + h;
        if (h < p.H) {
#pragma unroll
          for (int j = 0; j < S::COLS; ++j)
            if (c0 + j < n_rows) {
              float* q = dst + static_cast<int64_t>(j) * p.H;
              *q = p.acc_add ? *q + z[j] : z[j];
            }
        }
      }
    }
    if constexpr (MODE == CE_LSE) {
      // join the warp's lanes, then the quarters
      float2* s_part = reinterpret_cast<float2*>(smem + S::PARAM_OFFSET);
      __syncwarp();
      asm volatile("bar.sync %0, %1;" ::"r"(CE_BAR_EPI), "r"(S::EPI_WARPS * 32) : "memory");   // s_row has been read
#pragma unroll
      for (int j = 0; j < S::COLS; ++j) {
        if (j % 8 == 0 && c0 + j >= n_rows) break;
        float top = m[j];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        float t = sum[j] * exp_below(m[j], top);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
        if (lane == 0) s_part[quarter * NT + c0 + j] = make_float2(top, t);
      }
      __syncwarp();
      asm volatile("bar.sync %0, %1;" ::"r"(CE_BAR_EPI), "r"(S::EPI_WARPS * 32) : "memory");
      const int i = static_cast<int>(threadIdx.x) - 64;
      if (i < n_rows && i < NT) {
        float2 a = s_part[i];
        for (int q = 1; q < 4; ++q) {
          const float2 b = s_part[q * NT + i];
          const float top = fmaxf(a.x, b.x);
          a = make_float2(top, a.y * exp_below(a.x, top) + b.y * exp_below(b.x, top));
        }
        p.part[blockIdx.x * p.pitch + i] = a;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, CE_FEW_BUFS * S::NB);
  }
}

// Joins the parts of each row: the CTA takes `width` rows (a power of two up to 32), its threads equal shares of the
// parts.  The loss is (largest logit - target's) + log(sum), both at least 0, and not lse - target: that difference has lse's
// rounding, and left rows whose target is nearly certain with losses of some 1e-6 of either sign.
constexpr int CE_MERGE_THREADS = 512;
__global__ void __launch_bounds__(CE_MERGE_THREADS) k_ce_merge(const CeParams p, int parts, int width, float* loss, float* lse) {
  __shared__ float2 s[CE_MERGE_THREADS];
  const int r = threadIdx.x % width, share = threadIdx.x / width, shares = CE_MERGE_THREADS / width;
  const int row = blockIdx.x * width + r;
  float m = -INFINITY, sum = 0.0f;
  auto join = [&](float2 o) {
    const float m_new = fmaxf(m, o.x);
    const float base = m_new == -INFINITY ? 0.0f : m_new;
    sum = sum * exp_below(m, base) + o.y * exp_below(o.x, base);
    m = m_new;
  };
  ce_wait_before();
  if (blockIdx.x == 0) ce_join(p, threadIdx.x, CE_MERGE_THREADS);
  if (row < p.rows) {
#pragma unroll 8
    for (int i = share; i < parts; i += shares) join(__ldcs(p.part + i * p.pitch + row));
  }
  s[threadIdx.x] = make_float2(m, sum);
  for (int o = shares / 2; o > 0; o >>= 1) {
    __syncthreads();
    if (share < o) {
      join(s[threadIdx.x + o * width]);
      s[threadIdx.x] = make_float2(m, sum);
    }
  }
  if (share == 0 && row < p.rows) {
    const float rest = logf(sum);
    lse[row] = m + rest;
    const int64_t y = ce_target(p, row);
    float l = 0.0f;
    if (y >= p.V) {
      l = NAN;
      atomicOr(&p.meta->error, ERR_TARGET_RANGE);
    } else if (y >= 0) {
      l = (m - p.zy[row]) + rest;
    }
    loss[row] = l;
  }
}

// Shares of the vocabulary in dx, from the rows that take part: of the numbers whose parts there is room for, the one that
// deals the K steps out best to `workers` CTAs (or pairs).  Counted in K steps (about 0.27 us): a share's start and end, and its part of dx, written and read back
// (1072 x 2048 values in 15 parts took 48 us to add up; 3 parts leave 10, and the product 10 us longer).
constexpr int CE_SHARE_STEPS = 8;
constexpr float CE_PART_STEPS = 4.4e-6f;   // per value of dx: 8 bytes at 6.8 TB/s
__host__ __device__ __forceinline__ float ce_share_cost(int s, int n, int H, int tile, int steps, int workers) {
  const int64_t units = static_cast<int64_t>((n + tile - 1) / tile) * ((H + tile - 1) / tile);
  const int64_t waves = (units * s + workers - 1) / workers;
  return static_cast<float>(waves * ((steps + s - 1) / s + CE_SHARE_STEPS)) +
         (s > 1 ? static_cast<float>(s) * CE_PART_STEPS * static_cast<float>(n) * static_cast<float>(H) : 0.0f);
}
// What there is room for; one share needs none, or (several pieces) has it.
__host__ __device__ __forceinline__ int ce_most_shares(int most, int n, int H, int64_t room) {
  const int64_t fit = room / (static_cast<int64_t>(n > 0 ? n : 1) * H);
  return fit < 1 ? 1 : fit < most ? static_cast<int>(fit) : most;
}
__device__ __forceinline__ int ce_splits(int n, int H, int tile, int steps, int workers, int most) {   // a warp; most <= 32
  const int s = 1 + (threadIdx.x & 31);
  const float c = ce_share_cost(s, n, H, tile, steps, workers);
  const uint32_t cost = s <= most && s <= steps ? __float_as_uint(c) : 0x7F800000u;   // in the order of the floats
  const uint32_t least = __reduce_min_sync(0xFFFFFFFFu, cost);
  return max(1, __ffs(__ballot_sync(0xFFFFFFFFu, cost == least)));
}
struct CePack {
  const uint4* x;
  uint4* xp;
  int32_t* row_map;
  int T, t_pad;
  int dx_tile, dx_workers, dx_most;   // ce_splits
  int64_t dx_room;                    // elements of dx's parts
};
__device__ __forceinline__ void ce_put_meta(const CeParams& p, const CePack& q, int n, bool bad, float gain) {   // warp 0
  const int splits = ce_splits(n, p.H, q.dx_tile, p.piece_steps, q.dx_workers, ce_most_shares(q.dx_most, n, p.H, q.dx_room));
  if (threadIdx.x == 0) {
    p.meta->n = n;
    p.meta->error = bad ? ERR_TARGET_RANGE : 0u;
    p.meta->splits = splits;
    p.meta->gain = gain;
  }
}
// The rows that take part, packed in order: row_map[i] and xp[i] = x[row_map[i]] for i < n, zeros up to t_pad; dx of the
// other rows is zero.  Every CTA counts all targets (they are in the L2 after the first) and packs its share of the rows:
// one CTA that wrote the map for a second kernel took 19 us for 16384 rows, and 15 more for the copy.
constexpr int CE_PREP_THREADS = 1024;
__global__ void __launch_bounds__(CE_PREP_THREADS) k_ce_prep(const CeParams p, const CePack q) {
  __shared__ int s_warp[3][32];
  __shared__ uint32_t s_gain[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  ce_dependents();
  const int per = (q.T + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
  const int r0 = min(q.T, static_cast<int>(blockIdx.x) * per), r1 = min(q.T, r0 + per);
  int all = 0, ahead = 0, bad = 0;
  CeGain gain;
#pragma unroll 4
  for (int t = threadIdx.x; t < q.T; t += CE_PREP_THREADS) {
    const int64_t y = ce_target(p, t);
    const int in = y >= 0 && y < p.V;
    if (in && blockIdx.x == 0) gain.add(p, t);
    all += in;
    ahead += t < r0 ? in : 0;
    bad |= y >= p.V;
  }
  all = __reduce_add_sync(0xFFFFFFFFu, all);
  ahead = __reduce_add_sync(0xFFFFFFFFu, ahead);
  bad = __any_sync(0xFFFFFFFFu, bad);
  gain.join_warp();
  if (lane == 0) {
    s_gain[0][warp] = gain.loss;
    s_gain[1][warp] = gain.lse;
    s_warp[0][warp] = all;
    s_warp[1][warp] = ahead;
    s_warp[2][warp] = bad;
  }
  __syncthreads();
  const int n = __reduce_add_sync(0xFFFFFFFFu, s_warp[0][lane]);
  int at = __reduce_add_sync(0xFFFFFFFFu, s_warp[1][lane]);
  bad = __any_sync(0xFFFFFFFFu, s_warp[2][lane]);
  if (blockIdx.x == 0 && warp == 0) {
    gain.loss = s_gain[0][lane];
    gain.lse = s_gain[1][lane];
    gain.join_warp();
    ce_put_meta(p, q, n, bad != 0, gain.value());
  }
  const int per_row = p.H / 8;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  // 32 rows at a time: every warp knows which of them take part; the threads share out their pieces
  for (int t0 = r0; t0 < r1; t0 += 32) {
    const int t = t0 + lane;
    const int64_t y = t < r1 ? ce_target(p, t) : -1;
    const uint32_t in = __ballot_sync(0xFFFFFFFFu, y >= 0 && y < p.V);
    const int64_t pieces = static_cast<int64_t>(min(32, r1 - t0)) * per_row;
#pragma unroll 4
    for (int64_t e = threadIdx.x; e < pieces; e += CE_PREP_THREADS) {
      const int r = static_cast<int>(e / per_row);
      const int64_t src = t0 + r, c = e - static_cast<int64_t>(r) * per_row;
      if ((in >> r) & 1u) {
        const int64_t i = at + __popc(in & ((1u << r) - 1u));
        q.xp[i * per_row + c] = __ldcs(q.x + src * per_row + c);
      } else {
        reinterpret_cast<uint4*>(p.dx)[src * per_row + c] = zero;
      }
    }
    if (warp == 0 && (in >> lane) & 1u) q.row_map[at + __popc(in & ((1u << lane) - 1u))] = t;
    at += __popc(in);
  }
  for (int64_t i = n + blockIdx.x * int64_t(32) + warp; i < q.t_pad; i += gridDim.x * int64_t(32))
    for (int c = lane; c < per_row; c += 32) q.xp[i * per_row + c] = zero;
}

// dx of the packed rows from their fp32 parts, added in a fixed order: a thread has four columns, of eight or more shares
// every eighth (38 in a row took 7 us for 5 x 1024 values).
constexpr int CE_DX_THREADS = 256;
__global__ void __launch_bounds__(CE_DX_THREADS) k_ce_dx(const CeParams p, int steps) {
  __shared__ float4 s_sum[CE_DX_THREADS];
  ce_wait_before();
  const bool as_is = p.rows > 0;              // rows that take no part are among them
  const int most = ce_shares(p);
  if (!as_is && most == 1) return;            // dx has been written
  const float gain = p.meta->gain;
  const int split_steps = (p.piece_steps + most - 1) / most;
  const int splits = (steps + split_steps - 1) / split_steps;   // of the first piece; a shorter last one has no more
  const int slices = splits >= 8 ? 8 : 1, width = CE_DX_THREADS / slices;
  const int slice = threadIdx.x / width, lane = threadIdx.x % width;
  const int per_row = p.H / 4;
  const int64_t total = static_cast<int64_t>(ce_rows(p)) * per_row;
  for (int64_t e0 = blockIdx.x * int64_t(width); e0 < total; e0 += gridDim.x * int64_t(width)) {
    const int64_t e = e0 + lane;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](float4 o) {
      v.x += o.x;
      v.y += o.y;
      v.z += o.z;
      v.w += o.w;
    };
    const int64_t i = e / per_row;
    const int c = static_cast<int>(e - i * per_row);
    if (e < total) {
      const float4* a = reinterpret_cast<const float4*>(p.acc) + i * per_row + c;
#pragma unroll 8
      for (int s = slice; s < splits; s += slices) add(__ldcs(a + s * total));
    }
    if (slices > 1) {
      __syncthreads();
      s_sum[threadIdx.x] = v;
      __syncthreads();
      if (slice == 0)
        for (int q = 1; q < slices; ++q) add(s_sum[q * width + lane]);
    }
    if (slice == 0 && e < total) {
      uint2 o = make_uint2(pack_bf16x2(v.x * gain, v.y * gain), pack_bf16x2(v.z * gain, v.w * gain));
      if (as_is && !ce_takes_part(p, i)) o = make_uint2(0u, 0u);
      reinterpret_cast<uint2*>(p.dx)[(as_is ? i : static_cast<int64_t>(p.row_map[i])) * per_row + c] = o;
    }
  }
}

// dw of a piece from its fp32 parts, added in order: a thread has four columns.
__global__ void __launch_bounds__(256) k_ce_dw(const CeParams p, uint16_t* dw) {
  ce_wait_before();
  const int64_t total = static_cast<int64_t>(p.vcols) * (p.H / 4);
  const float4* a = reinterpret_cast<const float4*>(p.acc_w);
  const float gain = p.meta->gain;
  for (int64_t e = blockIdx.x * int64_t(256) + threadIdx.x; e < total; e += gridDim.x * int64_t(256)) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int s = 0; s < p.dw_splits; ++s) {
      const float4 o = __ldcs(a + s * total + e);
      v.x += o.x;
      v.y += o.y;
      v.z += o.z;
      v.w += o.w;
    }
    reinterpret_cast<uint2*>(dw)[e] =
        make_uint2(pack_bf16x2(v.x * gain, v.y * gain), pack_bf16x2(v.z * gain, v.w * gain));
  }
}

// ---- host side -------------------------------------------------------------------------------

// bf16 [rows, cols] with `pitch` elements per row, boxes of box_cols x box_rows.
bool ce_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t pitch, int box_cols, int box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch) * 2};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool ce_kmajor(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t pitch, int box = CE_HALF) {
  return ce_map(m, base, rows, cols, pitch, CE_BK, box);
}
bool ce_mnmajor(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t pitch) {
  return ce_map(m, base, rows, cols, pitch, 64, CE_BK);
}
bool ce_store(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t pitch) {
  return ce_map(m, base, rows, cols, pitch, 32, 32);
}

struct CeDevice {
  int sms = 0;
  int pairs = 0;               // CTA pairs that run at the same time (0: none)
};

// Launch with programmatic dependence on the kernel before (all but a call's first) and, for pairs, clusters of two.
template <typename... Params, typename... Args>
cudaError_t ce_go(void (*kernel)(Params...), int64_t grid, int threads, size_t smem, cudaStream_t stream, bool first,
                  bool pair, Args... args) {
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (!first) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (pair) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = 2;
    attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
template <int MODE, int CG, int STAGES>
bool ce_prepare() {
  return cudaFuncSetAttribute(k_ce_gemm<MODE, CG, STAGES>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              ce_smem_bytes(STAGES)) == cudaSuccess;
}
template <int MODE>
bool ce_prepare_few() {
  auto set = [](auto kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
  };
  bool ok = set(k_ce_few<MODE, 16>, FewShape<MODE, 16>::SMEM_BYTES) &&
            set(k_ce_few<MODE, 32>, FewShape<MODE, 32>::SMEM_BYTES);
  if constexpr (MODE != CE_LSE) ok = ok && set(k_ce_few<MODE, 64>, FewShape<MODE, 64>::SMEM_BYTES);
  return ok;
}
bool ce_device(CeDevice* out) {
  static CeDevice info[64];
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  std::lock_guard<std::mutex> lock(mu);
  CeDevice& d = info[dev];
  if (d.sms == 0) {
    int sms = 0, pairs = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) return false;
    constexpr int ST = CE_STAGES;
    if (!ce_prepare<CE_LSE, 1, ST>() || !ce_prepare<CE_DZ, 1, ST>() || !ce_prepare<CE_DW, 1, ST>() ||
        !ce_prepare<CE_DX, 1, ST>() || !ce_prepare<CE_LSE, 2, ST>() || !ce_prepare<CE_DZ, 2, ST>() ||
        !ce_prepare<CE_DW, 2, ST>() || !ce_prepare<CE_DX, 2, ST>() || !ce_prepare<CE_DW, 1, CE_SHORT>() ||
        !ce_prepare_few<CE_LSE>() || !ce_prepare_few<CE_DZ>() || !ce_prepare_few<CE_DX>())
      return false;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(128, 1, 1);
    cfg.blockDim = dim3(CE_THREADS, 1, 1);
    cfg.dynamicSmemBytes = ce_smem_bytes(ST);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&pairs, k_ce_gemm<CE_LSE, 2, ST>, &cfg) != cudaSuccess) {
      cudaGetLastError();   // clear: single CTAs are used instead
      pairs = 0;
    }
    d.pairs = pairs;
    d.sms = sms;
  }
  *out = d;
  return true;
}

template <int MODE>
cudaError_t ce_launch(bool pair, int64_t units, const CeDevice& dev, const CUtensorMap& a, const CUtensorMap& b,
                      const CUtensorMap& d, const CeParams& p, cudaStream_t stream, bool first, int* ctas = nullptr) {
  const int64_t grid = pair ? 2 * std::min<int64_t>(units, dev.pairs) : std::min<int64_t>(units, dev.sms);
  if (ctas != nullptr) *ctas = static_cast<int>(grid);
  return ce_go(pair ? k_ce_gemm<MODE, 2, CE_STAGES> : k_ce_gemm<MODE, 1, CE_STAGES>, grid, CE_THREADS,
               ce_smem_bytes(CE_STAGES), stream, first, pair, a, b, d, p);
}

int few_rows(int64_t T) { return T <= 16 ? 16 : T <= 32 ? 32 : 64; }   // NT of up to CE_FEW rows
template <int MODE>
cudaError_t ce_launch_few(int64_t T, int64_t units, const CeDevice& dev, const CUtensorMap& a, const CUtensorMap& b,
                          const CeParams& p, cudaStream_t stream, bool first, int* ctas = nullptr) {
  auto go = [&](auto nt, auto kernel) {
    using S = FewShape<MODE, decltype(nt)::value>;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(units, S::PER_SM * dev.sms));
    if (ctas != nullptr) *ctas = static_cast<int>(grid);
    return ce_go(kernel, grid, S::THREADS, S::SMEM_BYTES, stream, first, false, a, b, p);
  };
  const int nt = few_rows(T);
  if (nt == 16) return go(std::integral_constant<int, 16>{}, k_ce_few<MODE, 16>);
  if constexpr (MODE != CE_LSE) {               // (CE_LSE: up to CE_FEW_FWD rows)
    if (nt == 64) return go(std::integral_constant<int, 64>{}, k_ce_few<MODE, 64>);
  }
  return go(std::integral_constant<int, 32>{}, k_ce_few<MODE, 32>);
}

constexpr int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }
constexpr size_t up256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// Pairs compute tiles of 256 x 256, single CTAs tiles of 128 x 128, of which they take two in 1.6 times as long as a CTA of
// a pair its half tile (their operands are read twice as often).  Whichever is done first: forward 1000 x 1448 x 3600 with
// pairs 17.9 us, with single CTAs 23.7; 100 rows of it 15.9 and 13.9; 2000 x 512 x 500 10.9 and 8.6.
bool use_pair(const CeDevice& dev, int64_t m, int64_t n, int64_t splits = 1) {
  if (dev.pairs <= 0) return false;
  const int64_t pair = up(up(m, 256) * up(n, 256) * splits, dev.pairs) * 10;
  const int64_t single = up(up(m, 128) * up(n, 128) * splits, dev.sms) * 8;
  return pair <= single;
}

// Row tiles of a group: as many as keep their rows of A (of `bytes` each) within 48 MB of the L2.
int group_of(int64_t row_bytes, bool pair, int64_t most) {
  const int64_t g = (int64_t(48) << 20) / (row_bytes * (pair ? 256 : 128));
  return static_cast<int>(std::max<int64_t>(1, std::min(g, most)));
}

bool ce_sizes_ok(int64_t T, int64_t H, int64_t V) { return T >= 0 && H > 0 && V > 0; }
bool ce_sizes_supported(int64_t T, int64_t H, int64_t V) {
  return H % 8 == 0 && T <= (int64_t(1) << 24) && H <= (int64_t(1) << 20) && V <= (int64_t(1) << 28) &&
         up(T, 128) * up(V, 128) <= INT32_MAX / 2;
}
bool ce_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr size_t CE_MAX_CTAS = 1024;   // of a launch
struct CeFwdWs {
  size_t status, part, zy, total;
  int64_t pitch, parts;
};
CeFwdWs ce_fwd_ws(int64_t T, int64_t V) {
  CeFwdWs w{};
  w.pitch = up(T, 32) * 32;
  w.parts = 2 * up(V, 128);
  w.status = sizeof(CeMeta);
  w.part = w.status + CE_MAX_CTAS * sizeof(uint32_t);
  w.zy = up256(w.part + static_cast<size_t>(w.parts) * w.pitch * sizeof(float2));
  w.total = up256(w.zy + static_cast<size_t>(w.pitch) * sizeof(float));
  return w;
}

// Backward workspace: header, row map, packed (or cleared) x [t_pad, H], dz of one piece [t_pad, piece], fp32 parts of dx.
struct CeBwdWs {
  size_t status, row_map, xp, dz, acc, acc_w, total;
  int64_t t_pad, piece, pieces, room;   // room: elements of dx's parts
  int splits, dw_splits;
  bool few, as_is;             // as_is: rows are not packed (few rows never are)
};
constexpr int CE_MAX_SPLITS = 16;
// Rows as they are: packing is a launch of its own, 4 to 9 us with the choice of dx's shares, and saves products where rows
// take no part, which the host does not know; up to 512 rows and 2^33 products it is left out, where it saves hardly more than
// that with half of the rows masked.  dz's kernel copies x beside its products, which takes longer than these where H is
// large beside V.  As they are and packed, us with no rows masked, half of them, 80%:
//   100 x 1448 x 3600    28.4 33.5   28.4 32.4   28.4 32.0        512 x 1024 x 8192    44.1 47.7   43.8 43.0   43.7 38.7
//   400 x 1448 x 3600    35.7 41.1   35.5 38.3   35.4 36.4       1000 x 1448 x 3600    49.4 54.1   49.2 43.5   49.0 41.1
//   256 x 2048 x 16384   71.2 75.5   70.5 68.7   69.4 63.4       1024 x 1024 x 8192    54.8 58.8   54.3 50.0   53.8 41.1
//   100 x 2048 x 32000   92.3 99.8   92.4 96.1   91.9 94.5       1024 x 64 x 50257      110  111    110   77    110   61
// and 400 x 512 x 256, none masked, 21.9 and 16.2.
constexpr int64_t CE_AS_IS_ROWS = 512, CE_AS_IS_PRODUCTS = int64_t(1) << 33, CE_AS_IS_V = 1024;   // T, T * H * V, V
CeBwdWs ce_bwd_ws(int64_t T, int64_t H, int64_t V) {
  CeBwdWs w{};
  w.few = T <= CE_FEW;
  w.as_is = w.few || (T <= CE_AS_IS_ROWS && T * H <= CE_AS_IS_PRODUCTS / V &&
                       (V >= CE_AS_IS_V || 2 * H <= V));
  w.t_pad = w.few ? 2 * few_rows(T) : up(T, 256) * 256;   // few: dz and x twice
  auto entries = [&](int64_t elems) { return std::max(CE_MIN_PIECE, elems / std::max<int64_t>(w.t_pad, 256) / 256 * 256); };
  const int64_t most = w.few ? entries(CE_DZ_FEW)
                             : std::clamp(up(up(V, 2), 256) * 256, entries(CE_DZ_LEAST), entries(CE_DZ_MOST));
  w.pieces = up(V, most);
  w.piece = up(up(V, w.pieces), 256) * 256;
  w.pieces = up(V, w.piece);
  // dx has few tiles where there are few rows: its K is shared out
  const int64_t tiles = std::max<int64_t>(1, up(T, 128)) * up(H, 128);   // (no rows: no tiles)
  const int64_t wanted = w.few ? (T <= 32 ? 304 : 152) / tiles : tiles >= 8 * 152 ? 1 : CE_MAX_SPLITS;
  w.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(wanted, up(w.piece, 16 * CE_BK))));
  w.status = sizeof(CeMeta);
  w.row_map = w.status + CE_MAX_CTAS * sizeof(uint32_t);
  w.xp = up256(w.row_map + static_cast<size_t>(w.t_pad) * 4);
  w.dz = up256(w.xp + static_cast<size_t>(w.t_pad) * H * 2);
  w.acc = up256(w.dz + static_cast<size_t>(w.t_pad) * w.piece * 2);
  // dw has few tiles where the vocabulary and H are small: its rows are shared out
  const int64_t dw_tiles = up(w.piece, 128) * up(H, 128);
  w.dw_splits = w.few ? 1 : static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({CE_MAX_SPLITS, 152 / dw_tiles,
                                                                                     up(T, 8 * CE_BK)})));
  w.room = w.splits * T * H;
  if (!w.few) w.room = std::min(w.room, std::clamp(T * V / 8, CE_PARTS_LEAST, CE_PARTS_MOST));
  if (w.pieces > 1) w.room = std::max(w.room, T * H);
  else if (w.splits == 1) w.room = 0;
  w.acc_w = up256(w.acc + static_cast<size_t>(w.room) * 4);
  w.total = up256(w.acc_w + (w.dw_splits > 1 ? static_cast<size_t>(w.dw_splits) * w.piece * H * 4 : 0));
  return w;
}

}  // namespace
}  // namespace mx

using namespace mx;

extern "C" {

size_t linear_cross_entropy_workspace_size(int64_t T, int64_t H, int64_t V) {
  if (!ce_sizes_ok(T, H, V) || !ce_sizes_supported(T, H, V)) return 0;
  return ce_fwd_ws(T, V).total;
}

int linear_cross_entropy_fwd(const void* x, const void* w, const void* targets, int wide_targets, int64_t T, int64_t H,
                             int64_t V, float* loss, float* lse, void* workspace, size_t workspace_bytes,
                             void* stream) {
  if (!ce_sizes_ok(T, H, V) || wide_targets < 0 || wide_targets > 1) return MXFP8_ERR_INVALID_ARG;
  if (!ce_sizes_supported(T, H, V)) return MXFP8_ERR_UNSUPPORTED;
  if (workspace == nullptr) return MXFP8_ERR_INVALID_ARG;
  const CeFwdWs ws = ce_fwd_ws(T, V);
  if (!ce_aligned(workspace, 256) || workspace_bytes < ws.total) return MXFP8_ERR_WORKSPACE;
  if (T > 0) {
    if (x == nullptr || w == nullptr || targets == nullptr || loss == nullptr || lse == nullptr)
      return MXFP8_ERR_INVALID_ARG;
    if (!ce_aligned(x, 16) || !ce_aligned(w, 16) || !ce_aligned(targets, wide_targets ? 8 : 4) || !ce_aligned(loss, 4) ||
        !ce_aligned(lse, 4))
      return MXFP8_ERR_INVALID_ARG;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  if (T == 0) return cudaMemsetAsync(workspace, 0, sizeof(CeMeta), st) == cudaSuccess ? MXFP8_OK : MXFP8_ERR_CUDA;
  CeDevice dev;
  if (!ce_device(&dev)) return MXFP8_ERR_CUDA;
  const bool few = T <= CE_FEW_FWD;
  const bool pair = !few && use_pair(dev, T, V);
  const int64_t tile = pair ? 256 : 128;
  CeParams p{};
  p.meta = reinterpret_cast<CeMeta*>(base);
  p.rows = static_cast<int>(T);
  p.V = p.vcols = static_cast<int>(V);
  p.H = static_cast<int>(H);
  p.group_m = group_of(H * 2, pair, up(T, tile));
  p.status = reinterpret_cast<uint32_t*>(base + ws.status);
  p.targets = targets;
  p.wide_targets = wide_targets;
  p.part = reinterpret_cast<float2*>(base + ws.part);
  p.zy = reinterpret_cast<float*>(base + ws.zy);
  p.pitch = ws.pitch;
  p.timeout_ns = pipeline_wait_ns();
  CUtensorMap a, b;
  if (!ce_kmajor(&a, x, T, H, H, few ? few_rows(T) : CE_HALF) || !ce_kmajor(&b, w, V, H, H)) return MXFP8_ERR_CUDA;
  int ctas = 0;
  const cudaError_t e = few ? ce_launch_few<CE_LSE>(T, up(V, 128), dev, b, a, p, st, true, &ctas)
                            : ce_launch<CE_LSE>(pair, up(T, tile) * up(V, tile), dev, a, b, a, p, st, true, &ctas);
  if (e != cudaSuccess) return MXFP8_ERR_CUDA;
  p.join = p.status;
  p.joins = ctas;
  const int parts = few ? ctas : static_cast<int>(2 * up(V, tile));
  // as many rows per CTA as leave every SM one: 1531 rows of 394 parts took 14.8 us with 32
  int width = 32;
  while (width > 1 && up(T, width) < dev.sms) width /= 2;
  return ce_go(k_ce_merge, up(T, width), CE_MERGE_THREADS, 0, st, false, false, p, parts, width, loss, lse) ==
                 cudaSuccess
             ? MXFP8_OK
             : MXFP8_ERR_CUDA;
}

size_t linear_cross_entropy_bwd_workspace_size(int64_t T, int64_t H, int64_t V) {
  if (!ce_sizes_ok(T, H, V) || !ce_sizes_supported(T, H, V)) return 0;
  return ce_bwd_ws(T, H, V).total;
}

int linear_cross_entropy_bwd(const float* dloss, const float* dlse, const void* x, const void* w, const void* targets,
                             int wide_targets, const float* lse, int64_t T, int64_t H, int64_t V, void* dx, void* dw,
                             void* workspace, size_t workspace_bytes, void* stream) {
  if (!ce_sizes_ok(T, H, V) || wide_targets < 0 || wide_targets > 1) return MXFP8_ERR_INVALID_ARG;
  if (!ce_sizes_supported(T, H, V)) return MXFP8_ERR_UNSUPPORTED;
  if (workspace == nullptr || dw == nullptr || !ce_aligned(dw, 16)) return MXFP8_ERR_INVALID_ARG;
  const CeBwdWs ws = ce_bwd_ws(T, H, V);
  if (!ce_aligned(workspace, 256) || workspace_bytes < ws.total) return MXFP8_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {   // sums over no rows
    return cudaMemsetAsync(workspace, 0, sizeof(CeMeta), st) == cudaSuccess &&
                   cudaMemsetAsync(dw, 0, static_cast<size_t>(V) * H * 2, st) == cudaSuccess
               ? MXFP8_OK
               : MXFP8_ERR_CUDA;
  }
  for (const void* q : {x, w, static_cast<const void*>(dx)})
    if (q == nullptr || !ce_aligned(q, 16)) return MXFP8_ERR_INVALID_ARG;
  if (targets == nullptr || !ce_aligned(targets, wide_targets ? 8 : 4)) return MXFP8_ERR_INVALID_ARG;
  if (dloss == nullptr || lse == nullptr || !ce_aligned(dloss, 4) || !ce_aligned(lse, 4) || !ce_aligned(dlse, 4))
    return MXFP8_ERR_INVALID_ARG;
  CeDevice dev;
  if (!ce_device(&dev)) return MXFP8_ERR_CUDA;
  uint8_t* base = static_cast<uint8_t*>(workspace);
  uint16_t* xp = reinterpret_cast<uint16_t*>(base + ws.xp);
  uint16_t* dz = reinterpret_cast<uint16_t*>(base + ws.dz);
  CeParams p{};
  p.meta = reinterpret_cast<CeMeta*>(base);
  p.row_map = reinterpret_cast<int32_t*>(base + ws.row_map);
  p.V = static_cast<int>(V);
  p.H = static_cast<int>(H);
  p.targets = targets;
  p.wide_targets = wide_targets;
  p.lse = lse;
  p.dloss = dloss;
  p.dlse = dlse;
  p.acc_w = ws.dw_splits > 1 ? reinterpret_cast<float*>(base + ws.acc_w) : nullptr;
  p.dw_splits = ws.dw_splits;
  p.dx = static_cast<uint16_t*>(dx);
  p.timeout_ns = pipeline_wait_ns();
  const bool dx_pair = !ws.few && use_pair(dev, T, H, ws.splits);
  p.piece_steps = static_cast<int>(up(ws.piece, CE_BK));
  p.splits = ws.splits;
  if (ws.as_is) {
    p.rows = static_cast<int>(T);
    p.t_pad = static_cast<int>(ws.t_pad);
    p.dw_rows = static_cast<int>(ws.few ? ws.t_pad : T);
    if (!ws.few) {
      float least = INFINITY;
      const int most = std::min(p.piece_steps, ce_most_shares(ws.splits, p.rows, p.H, ws.room));
      for (int s = 1; s <= most; ++s) {
        const float c = ce_share_cost(s, p.rows, p.H, dx_pair ? 256 : 128, p.piece_steps, dx_pair ? dev.pairs : dev.sms);
        if (c < least) {
          least = c;
          p.splits = s;
        }
      }
    }
  } else {
    CePack q{};
    q.x = static_cast<const uint4*>(x);
    q.xp = reinterpret_cast<uint4*>(xp);
    q.row_map = reinterpret_cast<int32_t*>(base + ws.row_map);
    q.T = static_cast<int>(T);
    q.t_pad = static_cast<int>(ws.t_pad);
    q.dx_tile = dx_pair ? 256 : 128;
    q.dx_workers = dx_pair ? dev.pairs : dev.sms;
    q.dx_most = ws.splits;
    q.dx_room = ws.room;
    if (ce_go(k_ce_prep, std::min<int64_t>(up(T, 8), 2 * dev.sms), CE_PREP_THREADS, 0, st, true, false, p, q) != cudaSuccess)
      return MXFP8_ERR_CUDA;
  }
  p.acc = ws.pieces > 1 || p.splits > 1 ? reinterpret_cast<float*>(base + ws.acc) : nullptr;
  CUtensorMap x_k, x_mn, w_k, w_mn, dz_k, dz_mn, dz_st;
  p.dz = dz;
  p.dz_pitch = ws.piece;
  if (!ce_kmajor(&x_k, ws.as_is ? x : xp, ws.as_is ? T : ws.t_pad, H, H, ws.few ? few_rows(T) : CE_HALF) ||
      !ce_mnmajor(&x_mn, xp, ws.t_pad, H, H) || !ce_kmajor(&w_k, w, V, H, H) || !ce_mnmajor(&w_mn, w, V, H, H) ||
      !ce_kmajor(&dz_k, dz, ws.t_pad, ws.piece, ws.piece, ws.few ? 2 * few_rows(T) : CE_HALF) ||
      !ce_mnmajor(&dz_mn, dz, ws.t_pad, ws.piece, ws.piece) || !ce_store(&dz_st, dz, ws.t_pad, ws.piece, ws.piece))
    return MXFP8_ERR_CUDA;
  for (int64_t i = 0; i < ws.pieces; ++i) {
    const int64_t v0 = i * ws.piece, cols = std::min(ws.piece, V - v0);
    p.v0 = static_cast<int>(v0);
    p.vcols = static_cast<int>(cols);
    p.acc_add = i > 0;
    p.last = i + 1 == ws.pieces;
    const bool dz_pair = use_pair(dev, T, cols), dw_pair = use_pair(dev, cols, H, ws.dw_splits);
    const int64_t zt = dz_pair ? 256 : 128, wt = dw_pair ? 256 : 128, xt = dx_pair ? 256 : 128;
    p.group_m = group_of(H * 2, dz_pair, up(T, zt));
    p.d_rows = static_cast<int>(ws.t_pad);
    p.d_cols = static_cast<int>(ws.piece);
    const bool first = ws.as_is && i == 0;         // of the call's kernels
    CeParams z = p;
    if (first) {
      z.x = static_cast<const uint4*>(x);
      z.xp = reinterpret_cast<uint4*>(xp);
      z.status = reinterpret_cast<uint32_t*>(base + ws.status);
    }
    if ((ws.few ? ce_launch_few<CE_DZ>(T, up(cols, 128), dev, w_k, x_k, z, st, first, &p.joins)
                : ce_launch<CE_DZ>(dz_pair, up(T, zt) * up(cols, zt), dev, x_k, w_k, dz_st, z, st, first, &p.joins)) !=
        cudaSuccess)
      return MXFP8_ERR_CUDA;
    p.join = z.status;
    p.group_m = 1;
    // dx first: few rows leave w in the L2 for it, which dw overwrites
    if ((ws.few ? ce_launch_few<CE_DX>(T, up(H, 128) * p.splits, dev, w_mn, dz_k, p, st, false)
                : ce_launch<CE_DX>(dx_pair, up(T, xt) * up(H, xt) * p.splits, dev, dz_k, w_mn, dz_st, p, st, false)) !=
        cudaSuccess)
      return MXFP8_ERR_CUDA;
    CUtensorMap dw_st;
    if (!ce_store(&dw_st, static_cast<uint16_t*>(dw) + v0 * H, cols, H, H)) return MXFP8_ERR_CUDA;
    p.d_rows = static_cast<int>(cols);
    p.d_cols = static_cast<int>(H);
    // few K steps: a tile is mostly its epilogue, so two CTAs per SM; of more rows only where these are done in two turns
    // (256 x 2048 x 50257: 183 us with them, 162 without; 100 x 1448 x 3600: 33 and 37)
    const bool dw_short =
        ws.few || (T <= 4 * CE_BK && ws.dw_splits == 1 && up(cols, 128) * up(H, 128) <= 4 * dev.sms);
    const cudaError_t e =
        dw_short ? ce_go(k_ce_gemm<CE_DW, 1, CE_SHORT>, std::min<int64_t>(up(cols, 128) * up(H, 128), 2 * dev.sms),
                       CE_THREADS, ce_smem_bytes(CE_SHORT), st, false, false, dz_mn, x_mn, dw_st, p)
               : ce_launch<CE_DW>(dw_pair, up(cols, wt) * up(H, wt) * ws.dw_splits, dev, dz_mn, x_mn, dw_st, p, st,
                                   false);
    if (e != cudaSuccess) return MXFP8_ERR_CUDA;
    if (p.acc_w != nullptr && ce_go(k_ce_dw, std::min<int64_t>(up(cols * (H / 4), 256), 8 * dev.sms), 256, 0, st, false,
                                    false, p, static_cast<uint16_t*>(dw) + v0 * H) != cudaSuccess)
      return MXFP8_ERR_CUDA;
  }
  if (p.acc != nullptr && (ws.few || !ws.as_is || p.splits > 1) &&   // (otherwise dx has been written)
      ce_go(k_ce_dx, std::min<int64_t>(up(T * (H / 4), CE_DX_THREADS / 8), 8 * dev.sms), CE_DX_THREADS, 0, st, false, false, p,
            static_cast<int>(up(std::min(ws.piece, V), CE_BK))) != cudaSuccess)
    return MXFP8_ERR_CUDA;
  return MXFP8_OK;
}

}  // extern "C"

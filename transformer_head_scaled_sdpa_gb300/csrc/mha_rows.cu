// mha_rows.cu -- attention of a few query rows per sequence over a key/value
// cache: the decode step over the 8-bit cache and the step of a tree of
// drafted tokens over either cache, on the 5th-generation tensor cores,
// sm_103a.
//
// For each sequence b and key head the R = T * G rows (T drafted tokens, G
// query heads sharing the key head; T = G = 1 is a plain decode step) attend
// to the cached keys that the prefix length and the tree mask let them see:
//   s_jr = scale * k_j . q_r,  o_r = sum_j softmax_j(s_jr) v_j
// ("Attention Is All You Need", Section 3.2.1, Equation (1)).  The work is
// reading the cache once; a few rows leave most of a 128-row query tile empty,
// so both products are taken transposed, with the keys (then the features) as
// the 128 rows of the tensor-core tile and the query rows as its columns:
//   S^T [128 keys x R]     = K [128 keys x d]   Q^T
//   O^T [d x R]           += V^T [d x 128 keys] P^T [128 keys x R]
// K and V tiles are the A operands straight from shared memory as TMA wrote
// them (K rows along the reduction, V read transposed); one softmax thread
// owns one key (one TMEM lane) and finds all rows' scores of that key in its
// columns, so the key's scales and its visibility are per-thread values and
// the weights of a key are written as consecutive bytes.
//
// 8-bit cache: the e4m3 codes are the operands as they are (kind::f8f6f4), no
// unpacking pass.  The other operand is split into 8-bit pieces that add up
// to more than its own precision, one column per piece (columns are nearly
// free while reading the tiles bounds the tensor core):
//   q: two e4m3 pieces of q 2^-e (largest magnitude of the row in [128, 256)):
//      x1 = rn(x), x2 = rn(32 (x - x1)).  A bf16 value has 8 significant bits
//      and each piece holds 4 (and a sign), so x1 + x2 / 32 = x exactly down
//      to 2^-14, 2^-22 of the row's largest value.
//   p: three e5m2 pieces of the fp16 rounding of p; each takes 3 significant
//      bits of what is left, so the sum is p to 2^-11.  e5m2 has fp16's range,
//      so the pieces need no scales; weights are kept at 2^10 times their
//      reference, and what is lost below is 2^-27 of the reference.
//   v's scale 2^ev is folded into the weight: p_j = 2^(s_j + ev_j - m) with m
//      the row's largest s_j + ev_j, so that pieces are relative to the largest
//      contribution, and the denominator adds p_j 2^-ev_j.
// bf16 cache: kind::f16, q exact, p as two bf16 pieces (2^-15: the first is p
// cut to 8 bits, the second the rest rounded).
//
// Online softmax (scores in log2 units, q's factor scale * log2 e): the
// reference m of a row moves only when a tile's largest score exceeds it by
// more than a slack (8, or 5 for the 8-bit pieces' range); then O (in TMEM)
// and the sums are rescaled.  Sums are float32, one partial per thread and row,
// added up once at the end.
//
// Work: a unit is (split, sequence, key head, block of NR rows), with the key head
// and block the fastest: CTAs that run together read the rows of neighbouring
// heads, which lie side by side in the cache, and the same rows for their blocks
// (one head's rows alone are 128-byte pieces of DRAM pages: 161 us for 16
// sequences x 96 heads x 1,024 to 2,048 keys of 128 features in 8 bits when a CTA's
// work ran over consecutive heads, against 110).  rows_plan says how many splits
// there are, `balance` how they fall on the sequences of a ragged batch.  The grid
// has a CTA per unit, but CTAs are persistent: a running CTA cancels CTAs that have
// not started (cluster launch control) and takes their units, so the launch order
// balances the work (with equal static shares of the keys CTAs ended 25 % apart).
// A split of a sequence that has several leaves a partial (o, m, l) in the
// workspace, and rows_combine_kernel merges them exactly.
//
// Roles: one or two softmax warpgroups (thread = key = TMEM lane; they also prepare
// a CTA's first Q and write the outputs), one lane that issues every MMA, one that
// issues every TMA load, finds the units and publishes them to the others through a
// queue, over an 8-bit cache a warp that keeps the next tiles' scales in a ring, and
// one, two or four warps that prepare the next unit's Q pieces, output rows and mask
// words in a double buffer.  The MMA lane runs S(0), S(1), PV(0), S(2), PV(1), ...
// over all tiles of all units without a break at their borders: the next scores, and
// the loads of a whole ring, run during a unit's epilogue.  Every wait is bounded
// (abort flag, MHA_ERR_TIMEOUT).
//
// What bounds it (16 x 96 heads x 1,024 to 2,048 keys of 128 features in 8 bits, 610
// MB): 94 us, 6.5 TB/s, 0.95 of the measured copy; with 16 rows and 4 sequences (157
// MB) 36.5 us, 4.3 TB/s: the softmax threads' instructions (30 per weight: three pieces) and 384 units
// on 304 CTAs.  A unit costs five tiles of 128 keys beside its own (Q, the first
// maxima, the epilogue).  Code that runs for the first time costs some 30 cycles an
// instruction, so what a CTA runs before its first weights (10 to 20 thousand cycles)
// is kept short: loops where nothing else is lost, one site of each load and wait.
#include <cuda_bf16.h>

#include <type_traits>

#include "fp8.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace mha {
namespace {

constexpr int kScaleTiles = 8;     // tiles whose 8-bit scales are kept ahead
constexpr int kQueue = 4;          // published units
constexpr int kMaskWords = 4;      // 256 drafted tokens

template <bool F8_, int W_, int NR_>
struct RowsCfg {
  static constexpr bool F8 = F8_;
  static constexpr int W = W_;    // widest head
  static constexpr int NR = NR_;  // rows per unit
  static constexpr int EB = F8 ? 1 : 2;                  // bytes per cached element
  static constexpr int CHUNK = kKeys * 128;              // [128 keys x 128 B], 128-byte swizzle
  static constexpr int BLKS = W <= 128 ? 1 : 2;          // blocks of 128 features
  static constexpr int SLOT = kKeys * (W / BLKS) * EB;   // a ring slot: one block of a K or V tile
  static constexpr int QP = F8 ? 2 : 1;                  // pieces of q
  static constexpr int PP = F8 ? 3 : 2;                  // pieces of p
  // columns of S^T and O^T (multiples of 16: what is past the pieces is not read)
  static constexpr int NQ = QP * NR < 16 ? 16 : QP * NR;
  static constexpr int NP = (PP * NR + 15) / 16 * 16;
  static constexpr int Q_BYTES = NQ * W * EB;
  static constexpr int P_BYTES = kKeys * NP * EB;
  // barriers (512 bytes), units, scales, per-row values of two units and of the softmax
  static constexpr int SCALES = F8 ? kScaleTiles * kKeys * 2 : 0;
  static constexpr int MISC = 576 + 48 * kQueue + 16 + 160 + SCALES + 2 * (16 + 8 * kMaskWords) * NR + 24 * NR;
  static constexpr int FIXED = 2 * Q_BYTES + P_BYTES + MISC + 1024;
  // TMEM: S0 | S1 | O (per 128 features)
  static constexpr int M_O = W == 64 ? 64 : 128;         // rows of the O^T tile
  static constexpr uint32_t TM_S1 = NQ, TM_O = 2 * NQ;
  static constexpr uint32_t TM_USED = 2 * NQ + BLKS * NP;
  static constexpr uint32_t TMEM_COLS =
      TM_USED <= 32 ? 32 : (TM_USED <= 64 ? 64 : (TM_USED <= 128 ? 128 : (TM_USED <= 256 ? 256 : 512)));
  static_assert(TM_USED <= 512, "TMEM budget");
  // Two CTAs per SM when each can hold two tiles' worth of ring, else one with a deep
  // ring: one works while the other waits (8 bits, 96 heads x 1,024 to 2,048 keys: 16
  // sequences 99 us, one CTA 110; 4 with 16 drafted tokens 40 and 48; bf16, 64 features,
  // 32 x 8 heads x 30 to 280 keys with 12 drafted tokens 9.3 and 13.5).
  static constexpr int SLOTS2 = (115712 - FIXED) / SLOT;
  static constexpr bool TWO = SLOTS2 >= (BLKS == 1 ? 4 : 5) && NR <= 32 && TMEM_COLS <= 256;
  // Softmax warpgroups: two from 16 rows on, 32 where the CTA has the SM to itself (16
  // drafted tokens over 4 x 96 heads x 1,024 to 2,048 keys in 8 bits 40 us with two and
  // 43 with one; four of them for 64 rows of a bf16 cache 107 and 104, for 32 rows of 256
  // features in 8 bits 47.1 and 46.5).
  static constexpr int WGS = NR <= 8 || (NR <= 16 && !TWO) ? 1 : 2;
  static constexpr int RPT = NR / WGS;                   // rows per softmax thread
  // beside them: MMA, TMA, over an 8-bit cache scales, and Q; an 8-bit unit of many
  // rows has four warps for its Q's pieces (one: 27k cycles per unit of 64 rows)
  static constexpr bool MANY_Q = F8 && !TWO && WGS == 2;
  static constexpr int Q_THREADS = F8 ? (MANY_Q ? 128 : 32) : 64;
  static constexpr int THREADS = 128 * WGS + (MANY_Q ? 256 : 128);
  static constexpr int GW = RPT < 16 ? RPT : 16;         // rows handled together
  static constexpr int GROUPS = RPT / GW;
  static constexpr int SLOTS1 = (232448 - FIXED) / SLOT;
  static constexpr int SLOTS = TWO ? SLOTS2 : (SLOTS1 > 12 ? 12 : SLOTS1);
  static constexpr int MIN_BLOCKS = TWO ? 2 : 1;
  static_assert(SLOTS >= 2 * BLKS + 1, "ring: the next K tile while V waits");
  static constexpr int OFF_Q = SLOTS * SLOT;             // + buffer * Q_BYTES
  static constexpr int OFF_P = OFF_Q + 2 * Q_BYTES;
  static constexpr int OFF_MISC = OFF_P + P_BYTES;
  static constexpr int SMEM = OFF_MISC + MISC + 1024;
  static_assert(SMEM <= 232448, "shared memory");
  // barriers
  static constexpr int FULL = 0;              // + slot
  static constexpr int EMPTY = SLOTS;         // + slot
  static constexpr int Q_FULL = 2 * SLOTS;    // + buffer: Q and the unit's row values (Q_THREADS / 32 warps)
  static constexpr int Q_EMPTY = Q_FULL + 2;  // + buffer: the last scores and the epilogue are done
  static constexpr int S_FULL = Q_EMPTY + 2;  // + buffer
  static constexpr int P_FULL = S_FULL + 2;   // (every softmax warp)
  static constexpr int PV_DONE = P_FULL + 1;
  static constexpr int Q_FIRST = PV_DONE + 1;  // the first unit's Q (every softmax warp)
  static constexpr int O_FREE = Q_FIRST + 1;  // the epilogue has read O (every softmax warp)
  static constexpr int DRAIN = O_FREE + 1;
  static constexpr int SC_FULL = DRAIN + 1;            // + tile: scales (8-bit)
  static constexpr int SC_EMPTY = SC_FULL + (F8 ? kScaleTiles : 0);  // + tile: read (each softmax warp)
  static constexpr int UNIT_FULL = SC_EMPTY + (F8 ? kScaleTiles : 0);  // + queue slot: published
  static constexpr int UNIT_EMPTY = UNIT_FULL + kQueue;                // + queue slot: read (each consumer warp)
  static constexpr int CONSUMERS = 4 * WGS + 1 + (F8 ? 1 : 0) + Q_THREADS / 32;
  static constexpr int CLC = UNIT_EMPTY + kQueue;                      // a cancellation's response
  static constexpr int NBAR = CLC + 1;
  static constexpr int OFF_TMEM = OFF_MISC + 8 * NBAR;
  static constexpr int OFF_ABORT = OFF_TMEM + 4;
  static_assert(8 * NBAR + 8 <= 512 + 64, "barrier area");
  static constexpr int OFF_QUEUE = OFF_MISC + 576;       // Unit [kQueue], then the response (16 bytes)
  static constexpr int OFF_CLC = OFF_QUEUE + 48 * kQueue;
  static constexpr int OFF_TABLE = OFF_CLC + 16;  // sequences' first parts [33], tiles of a split (160 bytes)
  static constexpr int OFF_SCALES = OFF_TABLE + 160;  // [kScaleTiles][128]: k's byte, v's byte
  static constexpr int OFF_ROWS = OFF_SCALES + SCALES;
  // per buffer: factor, output row, lse index, live [NR each], mask words [NR][4]
  static constexpr int ROWS_BYTES = (16 + 8 * kMaskWords) * NR;
  static constexpr int OFF_SOFT = OFF_ROWS + 2 * ROWS_BYTES;  // reference, shift [NR each], red [NR][4]
  static_assert(OFF_Q % 1024 == 0 && OFF_P % 128 == 0 && OFF_MISC % 16 == 0 && ROWS_BYTES % 16 == 0, "alignment");
  static constexpr float SLACK = F8 ? 5.f : 8.f;         // reference moves beyond this (log2)
  static constexpr float LIFT = F8 ? 10.f : 0.f;         // weights are 2^LIFT at the reference
  // registers: the softmax warpgroups take from the others
  static constexpr bool SPLIT_REGS = TWO || WGS > 1;
  static constexpr int REGS_LAUNCH = 65536 / THREADS / (TWO ? 2 : 1) / 8 * 8;
  static constexpr int REGS_OTHER = MANY_Q ? 72 : (TWO && WGS == 2 ? 64 : 96);
  static constexpr int REGS_SOFT = MANY_Q ? 184 : (TWO ? (WGS == 2 ? 88 : 256 - REGS_OTHER) : 200);
  static_assert(!SPLIT_REGS || REGS_OTHER * (THREADS - 128 * WGS) + REGS_SOFT * 128 * WGS <= REGS_LAUNCH * THREADS,
                "register split");
};

// Shared-memory matrix descriptor without swizzle: core matrices of 8 rows x
// 16 bytes (128 contiguous bytes).
//   K-major operand (rows along M/N): lbo = bytes between 16-byte columns along
//     K, sbo = bytes between 8-row groups along M/N.
//   MN-major operand (rows along K): sbo = bytes between 16-byte columns along
//     M/N, lbo = bytes between 8-row groups along K.
__device__ __forceinline__ uint64_t smem_desc_plain(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) |
         (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (static_cast<uint64_t>(1) << 46);
}

// Instruction descriptor of kind::f8f6f4 with an e4m3 A, an e4m3 (0) or e5m2
// (1) B and a float32 accumulator (fields as idesc_bf16_f32).
constexpr uint32_t idesc_f8_f32(int M, int N, uint32_t b_format, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | (b_format << 10) | (static_cast<uint32_t>(a_mn_major) << 15) |
         (static_cast<uint32_t>(b_mn_major) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

template <bool F8>
__device__ __forceinline__ void umma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (F8) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  } else {
    umma_ss(d, a, b, idesc, acc);
  }
}

// True for every thread of a softmax warpgroup when any of them passes true
// (named barrier `id` over its 128 threads).
__device__ __forceinline__ bool any_of_128(uint32_t id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "r"(id)
      : "memory");
  return r != 0;
}

// Two fp16 values to e5m2 (nearest even); low half to bits 0-7.
__device__ __forceinline__ uint32_t half2_to_e5m2x2(uint32_t h2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(h2));
  return r;
}
// e5m2 is fp16 without its low byte.
__device__ __forceinline__ uint32_t e5m2x2_to_half2(uint32_t c) { return __byte_perm(c, 0, 0x1404); }
__device__ __forceinline__ uint32_t half2_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The larger magnitudes of pairs of bf16 (NaN loses).
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t m, uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a & 0x7fff7fffu), "r"(b & 0x7fff7fffu));
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(m));
  return r;
}

// Largest value of the warp.
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Sums of N values over the warp, N <= 32 a power of two: each step halves the
// values a lane keeps and adds its partner's for them.  Lane i returns the sum
// of value i / (32 / N).
template <int N>
__device__ __forceinline__ float warp_sums(const float (&v)[N], int lane) {
  float x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = v[i];
  int keep = N;
#pragma unroll
  for (int bit = 16; bit; bit >>= 1) {
    if (keep > 1) {
      keep >>= 1;
      const bool hi = (lane & bit) != 0;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        if (i >= keep) break;
        const float send = hi ? x[i] : x[i + keep];
        x[i] = (hi ? x[i + keep] : x[i]) + __shfl_xor_sync(0xffffffffu, send, bit);
      }
    } else {
      x[0] += __shfl_xor_sync(0xffffffffu, x[0], bit);
    }
  }
  return x[0];
}

// 8 or 16 consecutive 32-bit columns of this warp's TMEM lanes.
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t at, uint32_t (&r)[N]) {
  static_assert(N == 4 || N == 8 || N == 16, "columns");
  if constexpr (N == 16) {
    tmem_ld16(at, r);
  } else if constexpr (N == 4) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at));
  } else {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                   "=r"(r[7])
                 : "r"(at));
  }
}
template <int N>
__device__ __forceinline__ void tmem_st_cols(uint32_t at, const uint32_t (&r)[N]) {
  static_assert(N == 4 || N == 8 || N == 16, "columns");
  if constexpr (N == 16) {
    tmem_st16(at, r);
  } else if constexpr (N == 4) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
  } else {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(at),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
  }
}

// A position in the ring of K and V blocks.  A unit's are loaded in the order
// K(0) K(1) V(0) K(2) V(1) ... V(last).
template <int SLOTS>
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void advance() {
    if (++slot == SLOTS) {
      slot = 0;
      phase ^= 1;
    }
  }
};

template <bool F8, int W, int NR>
__global__ void __launch_bounds__((RowsCfg<F8, W, NR>::THREADS), (RowsCfg<F8, W, NR>::MIN_BLOCKS))
    rows_kernel(const __grid_constant__ RowsParams p) {
  using C = RowsCfg<F8, W, NR>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t s_base = smem_u32(smem);
  auto bar = [&](int id) { return s_base + C::OFF_MISC + 8u * static_cast<uint32_t>(id); };
  const uint32_t sP = s_base + C::OFF_P;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_TMEM);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
  Unit* queue = reinterpret_cast<Unit*>(smem + C::OFF_QUEUE);
  auto row_factor = [&](int buf) { return reinterpret_cast<float*>(smem + C::OFF_ROWS + buf * C::ROWS_BYTES); };
  auto row_out = [&](int buf) { return reinterpret_cast<int*>(smem + C::OFF_ROWS + buf * C::ROWS_BYTES) + NR; };
  auto row_lse = [&](int buf) { return reinterpret_cast<int*>(smem + C::OFF_ROWS + buf * C::ROWS_BYTES) + 2 * NR; };
  auto row_live = [&](int buf) { return reinterpret_cast<int*>(smem + C::OFF_ROWS + buf * C::ROWS_BYTES) + 3 * NR; };
  auto row_mask = [&](int buf) {
    return reinterpret_cast<uint64_t*>(smem + C::OFF_ROWS + buf * C::ROWS_BYTES + 16 * NR);
  };
  float* row_ref = reinterpret_cast<float*>(smem + C::OFF_SOFT);  // references less LIFT
  float* row_shift = row_ref + NR;
  float* red = row_shift + NR;  // [NR][4 warps]
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int tid = static_cast<int>(threadIdx.x);
  constexpr int SOFT = 128 * C::WGS;            // softmax threads
  constexpr int kMmaWarp = 4 * C::WGS, kLoadWarp = kMmaWarp + 1, kScaleWarp = kMmaWarp + 2;
  constexpr int kQWarp = kMmaWarp + (F8 ? 3 : 2);
  const int n_rows = p.T * p.G;
  const int blocks = (n_rows + NR - 1) / NR;    // blocks of rows per key head (the faster index of a unit)

  if (tid == 0) {
    for (int s = 0; s < C::SLOTS; ++s) {
      mbar_init(bar(C::FULL + s), 1);
      mbar_init(bar(C::EMPTY + s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::Q_FULL + i), C::Q_THREADS / 32);
      mbar_init(bar(C::Q_EMPTY + i), 1 + SOFT / 32);
      mbar_init(bar(C::S_FULL + i), 1);
    }
    mbar_init(bar(C::P_FULL), SOFT / 32);
    mbar_init(bar(C::PV_DONE), 1);
    mbar_init(bar(C::Q_FIRST), SOFT / 32);
    mbar_init(bar(C::O_FREE), SOFT / 32);
    mbar_init(bar(C::DRAIN), 1);
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(bar(C::UNIT_FULL + i), 1);
      mbar_init(bar(C::UNIT_EMPTY + i), C::CONSUMERS);
    }
    mbar_init(bar(C::CLC), 1);
    if constexpr (F8) {
      for (int i = 0; i < kScaleTiles; ++i) {
        mbar_init(bar(C::SC_FULL + i), 1);
        mbar_init(bar(C::SC_EMPTY + i), 4 * C::WGS);
      }
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();  // the barriers are set up
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), C::TMEM_COLS);
    tmem_relinquish();
    tc_fence_before();
  }
  if (warp == kLoadWarp) {
    // (this warp goes on to its loads without the tensor memory's address)
    asm volatile("barrier.cta.arrive 15, %0;" ::"n"(C::THREADS) : "memory");
  } else {
    asm volatile("barrier.cta.sync 15, %0;" ::"n"(C::THREADS) : "memory");
    tc_fence_after();
  }
  const uint32_t tmem = *tmem_slot;  // (not the load warp's, which did not wait)
  griddep_wait();  // global memory only from here on
  // the next launch may set itself up once every unit is taken (it waits for this
  // grid before it touches global memory) and every CTA has its tensor memory, which
  // the load warp does not know
  if (warp != kLoadWarp) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const bool ordered = longest_first(p, kSms * C::MIN_BLOCKS);
  const int blks = C::BLKS == 1 ? 1 : (p.d + 127) / 128;  // 128-feature blocks in use
  // The k-th published unit (each consumer warp takes each, in order); b = -1 at
  // the end of the work or when the CTA gave up.
  auto take = [&](int k, int site) {
    const int slot = k % kQueue;
    Unit w;
    if (!warp_wait(bar(C::UNIT_FULL + slot), (k / kQueue) & 1, abort_flag, site + C::UNIT_FULL + slot)) {
      w.b = -1;
      return w;
    }
    const int4* src = reinterpret_cast<const int4*>(queue + slot);
    int4* dst = reinterpret_cast<int4*>(&w);
#pragma unroll
    for (int i = 0; i < 3; ++i) dst[i] = src[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::UNIT_EMPTY + slot));
    return w;
  };
  // Phase of Q_FULL for unit k (the first unit has a barrier of its own).
  auto q_phase = [](int k) { return static_cast<uint32_t>(((k >> 1) - ((k & 1) ? 0 : 1)) & 1); };
  // Output row of row r of a unit (-1 past the last), t: its drafted token.
  auto out_row = [&](const Unit& it, int r, int* t) {
    const int gr = it.rb * NR + r;
    *t = -1;
    if (gr >= n_rows) return -1;
    *t = p.G == 1 ? gr : gr / p.G;
    return (it.b * p.T + *t) * p.H + it.hk * p.G + (gr - *t * p.G);
  };
  // Asks a unit's Q and mask words into L2.
  auto ask_q = [&](const Unit& it, int qt, int threads) {
#pragma unroll 1
    for (int r = qt >> 3; r < NR; r += threads >> 3) {
      int t;
      const int out = out_row(it, r, &t);
      if (out < 0) break;
      if (64 * (qt & 7) < p.d)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const uint16_t*>(p.q) +
                                                      static_cast<long long>(out) * p.d + 64 * (qt & 7)));
      if (p.tree_mask && (qt & 7) == 7)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.tree_mask +
                                                      (static_cast<long long>(it.b) * p.T + t) * p.words));
    }
  };
  // A unit's Q, output rows and mask words into buffer `buf`, by thread qt of a
  // multiple of 32 (eight threads per row); false when `buffer_free` gave up.
  auto prepare_q = [&](auto threads, const Unit& it, int buf, int qt, auto buffer_free) {
    constexpr int RP = decltype(threads)::value / 8;
    constexpr int PER = W / 64;                    // 16-byte pieces of a row per thread
    const int sub = qt & 7;
    const uint32_t sQ = s_base + C::OFF_Q + buf * C::Q_BYTES;
    if (NR < RP && (qt >> 3) >= NR) return buffer_free();  // (whole warps)
    auto load_row = [&](int r, int* t, uint4 (&v)[PER]) {
      const int out = out_row(it, r, t);
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                        static_cast<long long>(max(out, 0)) * p.d);
#pragma unroll
      for (int z = 0; z < PER; ++z) {
        // 8-bit: 16 elements to a thread, in two pieces; bf16: 8
        const int piece = F8 ? 2 * (sub + 8 * (z >> 1)) + (z & 1) : sub + 8 * z;
        v[z] = make_uint4(0, 0, 0, 0);
        if (out >= 0 && 8 * piece < p.d) v[z] = __ldg(src + piece);
      }
      return out;
    };
    uint4 v[PER], ahead[PER];
    int t, t_ahead = -1, out_ahead = -1;
    int out = load_row(qt >> 3, &t, v);
    if (!buffer_free()) return false;
#pragma unroll 1
    for (int rr = 0; rr < NR; rr += RP) {
      const int r = rr + (qt >> 3);
      if (rr + RP < NR) out_ahead = load_row(r + RP, &t_ahead, ahead);
      const bool live = t >= 0 && t < it.live;
      if (sub == 0) {
        row_out(buf)[r] = out;
        row_lse(buf)[r] = out < 0 ? 0 : (it.b * p.H + out % p.H) * p.T + t;
        row_live(buf)[r] = live;
      }
      if (sub < kMaskWords) {
        // (a chain's words: bits 0 .. t)
        uint64_t word = 0;
        if (live && p.tree_mask) {
          if (sub < p.words)
            word = __ldg(p.tree_mask + (static_cast<long long>(it.b) * p.T + t) * p.words + sub);
        } else if (live) {
          const int bits = t + 1 - 64 * sub;
          word = bits >= 64 ? ~0ull : (bits <= 0 ? 0ull : (1ull << bits) - 1);
        }
        row_mask(buf)[r * kMaskWords + sub] = word;
      }
      if constexpr (F8) {
        uint32_t top = 0;  // the largest magnitudes of even and odd elements (bf16 pair)
#pragma unroll
        for (int z = 0; z < PER; ++z)
          top = max_abs_bf16x2(max_abs_bf16x2(top, v[z].x, v[z].y), v[z].z, v[z].w);
        float amax = fmaxf(bf16_lo(top), bf16_hi(top));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        // q 2^-e with the largest magnitude in [128, 256)
        const int e = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 7, -100);
        const float inv = pow2i(-e);
        if (sub == 0) row_factor(buf)[r] = pow2i(e) * p.scale_log2;
        // (a loop over eight elements, the rest moving up: unrolled this was most of the
        // code that a CTA waits for before its first scores)
        uint32_t to = sQ + sub * (C::NQ * 16) + r * 16;
#pragma unroll 1
        for (int z = 0; z < PER; ++z) {
          const uint32_t q4[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
          uint32_t a[4], c2[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float x0 = bf16_lo(q4[x]) * inv, x1 = bf16_hi(q4[x]) * inv;
            a[x] = pack_e4m3x2(x0, x1);
            const uint32_t h2 = e4m3x2_to_half2(static_cast<uint16_t>(a[x]));
            c2[x] = pack_e4m3x2((x0 - half_lo(h2)) * 32.f, (x1 - half_hi(h2)) * 32.f);
          }
          st_shared_v2(to, a[0] | (a[1] << 16), a[2] | (a[3] << 16));
          st_shared_v2(to + NR * 16, c2[0] | (c2[1] << 16), c2[2] | (c2[3] << 16));
          // (the other half of the 16 elements, then the next 16 of the thread)
          to += (z & 1) ? 8 * (C::NQ * 16) - 8 : 8;
#pragma unroll
          for (int x = 0; x + 1 < PER; ++x) v[x] = v[x + 1];
        }
      } else {
#pragma unroll
        for (int z = 0; z < PER; ++z)
          st_shared_v4(sQ + (sub + 8 * z) * (C::NQ * 16) + r * 16, v[z].x, v[z].y, v[z].z, v[z].w);
      }
      out = out_ahead;
      t = t_ahead;
#pragma unroll
      for (int z = 0; z < PER; ++z) v[z] = ahead[z];
    }
    return true;
  };

  if (warp >= kMmaWarp) {
    if constexpr (C::SPLIT_REGS) regs_decrease<C::REGS_OTHER>();
    if (warp == kLoadWarp) {
      // ---- TMA producer (one lane)
      const int site = kRoleRowsLoad * 64;
      int* table = reinterpret_cast<int*>(smem + C::OFF_TABLE);
      if (balanced(p)) {
        int first, splits, per;
        balance(p, lane, &first, &splits, &per);
        if (lane < p.B) table[lane + 1] = first + splits;
        if (lane == 0) {
          table[0] = 0;
          table[p.B + 1] = per;
        }
        __syncwarp();
      } else if (ordered) {
        const int place = place_of(p, lane);
        if (lane < p.B) table[place] = lane;
        __syncwarp();
      }
      auto unit_at = [&](int index) {
        const int part = index / p.units;
        if (!balanced(p))
          return unit_of(p, index, blocks, ordered ? table[part] : part % p.B, part / p.B, 0);
        int b = 0;
        while (b < p.B && part >= table[b + 1]) ++b;
        if (b == p.B) {
          Unit none = {};
          return none;
        }
        return unit_of(p, index, blocks, b, part - table[b], table[p.B + 1]);
      };
      if (elect_one()) {
        Ring<C::SLOTS> ring;
        int loaded = 0;  // slots filled so far
        bool ok = true;
        // one tile of K or V: whole in boxes of 128 keys, a ragged one in boxes of
        // kBoxKeys as far as it goes
        auto load = [&](const CUtensorMap* big, const CUtensorMap* small, int key, int end, int hk, int b) {
          const int boxes = end - key >= kKeys ? 0 : (end - key + kBoxKeys - 1) / kBoxKeys;
          const uint32_t box_bytes = boxes == 0 ? kKeys * 128 : boxes * kBoxKeys * 128;
#pragma unroll 1
          for (int blk = 0; blk < C::BLKS; ++blk) {
            if (blk >= blks) break;
            const int s = ring.slot;
            ok = ok && (loaded < C::SLOTS ||
                        thread_wait(bar(C::EMPTY + s), ring.phase ^ 1, abort_flag, site + C::EMPTY + s));
            if (!ok) return;
            const int f0 = blk * 128;
            const int chunks = (min(p.d - f0, 128) * C::EB + 127) / 128;
            const uint32_t full = bar(C::FULL + s);
            mbar_arrive_expect_tx(full, chunks * box_bytes);
            for (int c = 0; c < chunks; ++c) {
              const uint32_t dst = s_base + s * C::SLOT + c * C::CHUNK;
              const int f = f0 + c * (128 / C::EB);
              if (boxes == 0) {
                tma_load_4d(dst, big, full, f, hk, key, b);
              } else {
                for (int x = 0; x < boxes; ++x)
                  tma_load_4d(dst + x * kBoxKeys * 128, small, full, f, hk, key + x * kBoxKeys, b);
              }
            }
            ++loaded;
            ring.advance();
          }
        };
        // The units: this CTA's own, then those of CTAs that have not started.  The
        // next is asked for half-way through a unit's loads and published as soon
        // as it is known, so that its Q and scales are there when its turn comes.
        volatile int never = 0;
        int published = 0;
        auto publish = [&](const Unit& w) {
          const int slot = published % kQueue;
          ok = ok && (published < kQueue ||
                      thread_wait(bar(C::UNIT_EMPTY + slot), ((published / kQueue) - 1) & 1, abort_flag,
                                  site + C::UNIT_EMPTY + slot));
          if (!ok) return;
          queue[slot] = w;
          mbar_arrive(bar(C::UNIT_FULL + slot));
          ++published;
        };
        uint32_t answers = 0;
        bool asked = false, done = false;
        Unit w = unit_at(static_cast<int>(blockIdx.x)), next = w;
        bool got = w.splits > 0;  // a unit to work on
        if (got) publish(w);
        while (ok) {
          const bool works = got;
          got = false;
          // the next unit, if its answer is there or `must` be waited for
          auto poll = [&](bool must) {
            while (!got && !done && ok) {
              if (!asked) {
                mbar_arrive_expect_tx(bar(C::CLC), 16);
                clc_try_cancel(s_base + C::OFF_CLC, bar(C::CLC));
                asked = true;
              }
              // (the response lands whatever happens: it is waited for even when giving up)
              if (must) ok = mbar_wait(bar(C::CLC), answers & 1, &never, p.status, site + C::CLC) && *abort_flag == 0;
              else if (!mbar_test(bar(C::CLC), answers & 1)) return;
              ++answers;
              asked = false;
              const int index = clc_query_first_ctaid_x(s_base + C::OFF_CLC);  // -1: none was left
              fence_proxy_async_smem();  // (the next response overwrites this one)
              done = index < 0;
              if (done || !ok) return;
              next = unit_at(index);
              got = next.splits > 0;
              if (got) publish(next);
            }
          };
          // K(0) K(1) V(0) K(2) V(1) ... V(last), then the next unit for certain
          const int n = works ? w.t1 - w.t0 : 0;
          for (int s = 0;; ++s) {
            if (s < 2 * n && ok) {
              const bool last = s == 2 * n - 1, v = last || (s > 0 && (s & 1) == 0);
              const int x = w.t0 + (last ? n - 1 : (v ? s / 2 - 1 : (s + 1) / 2));
              load(v ? &p.tm_v : &p.tm_k, v ? &p.tm_v_box : &p.tm_k_box, x * kKeys, w.end, w.hk, w.b);
            }
            const bool must = s >= 2 * n || !ok;
            if (s >= n || must) poll(must);
            if (must) break;
          }
          if (!got) break;
          w = next;
        }
        if (asked) mbar_wait(bar(C::CLC), answers & 1, &never, p.status, site + C::CLC);
        Unit end;
        end.b = -1;
        publish(end);
        // every copy started must land before the CTA exits
        for (int x = min(loaded, C::SLOTS); x > 0; --x) {
          // (the slot x before the next one)
          const int s = ring.slot >= x ? ring.slot - x : ring.slot - x + C::SLOTS;
          mbar_wait(bar(C::FULL + s), ring.slot >= x ? ring.phase : ring.phase ^ 1, &never, p.status, site + C::FULL + s);
        }
      }
      __syncwarp();
    } else if (warp == kMmaWarp) {
      // ---- MMA issuer (one lane): S(0) S(1) PV(0) S(2) PV(1) ... over all units' tiles
      const int site = kRoleRowsMma * 64;
      if (elect_one()) {
        constexpr int KSTEP = F8 ? 32 : 16;               // reduction elements per MMA
        const int n_ks = (p.d + KSTEP - 1) / KSTEP;
        constexpr int KS_BLK = 128 / KSTEP;               // steps of a 128-feature block
        constexpr uint32_t idesc_s = F8 ? idesc_f8_f32(128, C::NQ, 0, false, false)
                                        : idesc_bf16_f32(128, C::NQ, false, false);
        constexpr uint32_t idesc_o = F8 ? idesc_f8_f32(C::M_O, C::NP, 1, true, true)
                                        : idesc_bf16_f32(C::M_O, C::NP, true, true);
        // K: rows of 128 bytes per chunk, 8-row groups 1024 B apart, +32 B per step
        // inside a chunk.  V transposed: features contiguous in a 128-byte row, next
        // chunk of features CHUNK apart, 8-key groups 1024 B apart.
        const uint64_t dk0 = smem_desc_sw128(s_base, 16, 1024);
        const uint64_t dv0 = smem_desc_sw128(s_base, C::CHUNK, 1024);
        const uint64_t dq0 = smem_desc_plain(s_base + C::OFF_Q, C::NQ * 16, 128);
        const uint64_t dp0 = smem_desc_plain(sP, 128, kKeys * 16);
        bool ok = true;
        auto wait = [&](int id, uint32_t parity) { ok = ok && thread_wait(bar(id), parity, abort_flag, site + id); };
        // Scores run one tile ahead of the products.  A unit's blocks lie in the ring
        // in the order K(0) K(1) V(0) K(2) ... V(last): `k_at` and `v_at` count ring
        // items (tiles of K or V).
        uint32_t ts = 0, tp = 0;        // tiles whose scores, products are issued
        uint32_t k_at = 0, v_at = 0;
        int taken = 0, ks = -1, kp = -1;
        int s_n = 0, s_i = 0;           // the scores' unit: tiles, tiles issued
        int n_odd = 0, n_even = 0;      // tiles of odd and even units
        int p_n = 0, p_i = 0;           // the products' unit
        bool more = true, q_known = false;
        while (ok) {
          // ---- the next tile's scores; at a unit's border only if it and its Q are
          // there, unless nothing else is left to do
          if (more && ts < tp + 2) {
            const bool must = ts == tp;
            if (s_i == s_n) {
              const int slot = taken % kQueue;
              const uint32_t full = bar(C::UNIT_FULL + slot), parity = (taken / kQueue) & 1;
              if (must) wait(C::UNIT_FULL + slot, parity);
              if (ok && (must || mbar_test(full, parity))) {
                const int n = queue[slot].b < 0 ? -1 : queue[slot].t1 - queue[slot].t0;
                mbar_arrive(bar(C::UNIT_EMPTY + slot));
                ++taken;
                if (n == 0) continue;
                if (n < 0) {
                  more = false;
                } else {
                  s_n = n;
                  s_i = 0;
                  ++ks;
                  q_known = false;
                }
              }
            }
            if (s_i < s_n && !q_known) {
              const int id = ks == 0 ? C::Q_FIRST : C::Q_FULL + (ks & 1);
              const uint32_t parity = ks == 0 ? 0 : q_phase(ks);
              if (must) wait(id, parity);
              q_known = ok && (must || mbar_test(bar(id), parity));
            }
            if (q_known && s_i < s_n) {
              const uint64_t q = dq0 + static_cast<uint64_t>(((ks & 1) * C::Q_BYTES) >> 4);
              const uint32_t d = tmem + ((ts & 1) ? C::TM_S1 : 0u);
              uint32_t slot = 0;
#pragma unroll
              for (int blk = 0; blk < C::BLKS; ++blk) {
                if (blk >= blks) break;
                const uint32_t item = k_at * blks + blk;
                slot = item % C::SLOTS;
                wait(C::FULL + slot, (item / C::SLOTS) & 1);
                if (!ok) break;
                tc_fence_after();
                const uint64_t a = dk0 + static_cast<uint64_t>((slot * C::SLOT) >> 4);
#pragma unroll
                for (int x = 0; x < KS_BLK; ++x) {
                  const int step = blk * KS_BLK + x;
                  if (step < n_ks)
                    umma<F8>(d, a + static_cast<uint64_t>(((x >> 2) * C::CHUNK + (x & 3) * 32) >> 4),
                             q + static_cast<uint64_t>(step * 2 * C::NQ), idesc_s, step > 0 ? 1u : 0u);
                }
                if (blk < blks - 1) umma_commit(bar(C::EMPTY + slot));
              }
              if (!ok) break;
              umma_commit(bar(C::S_FULL + (ts & 1)));
              umma_commit(bar(C::EMPTY + slot));
              if (ks & 1) n_odd = s_n;
              else n_even = s_n;
              // (a last tile's K is followed by its own V, after the one before)
              k_at += s_i + 1 < s_n ? (s_i == 0 ? 1 : 2) : (s_n == 1 ? 2 : 3);
              ++s_i;
              if (s_i == s_n) umma_commit(bar(C::Q_EMPTY + (ks & 1)));
              ++ts;
              if (must) continue;
            }
          }
          if (tp == ts) {
            if (!more) break;
            continue;
          }
          // ---- O += V^T P^T of tile tp
          if (p_i == p_n) {
            ++kp;
            p_n = (kp & 1) ? n_odd : n_even;
            p_i = 0;
            // (O is free once the last unit's epilogue has read it)
            if (kp > 0) wait(C::O_FREE, (kp - 1) & 1);
            v_at += p_n == 1 ? 1 : 2;  // (from the unit's first item)
          }
          wait(C::P_FULL, tp & 1);
          uint32_t slot = 0;
#pragma unroll
          for (int blk = 0; blk < C::BLKS; ++blk) {
            if (blk >= blks) break;
            const uint32_t item = v_at * blks + blk;
            slot = item % C::SLOTS;
            wait(C::FULL + slot, (item / C::SLOTS) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem + C::TM_O + blk * C::NP;
            const uint64_t a = dv0 + static_cast<uint64_t>((slot * C::SLOT) >> 4);
#pragma unroll
            for (int step = 0; step < kKeys / KSTEP; ++step)
              umma<F8>(d, a + static_cast<uint64_t>((step * KSTEP * 128) >> 4),
                       dp0 + static_cast<uint64_t>((step * KSTEP * 16) >> 4), idesc_o,
                       (p_i > 0 || step > 0) ? 1u : 0u);
            if (blk < blks - 1) umma_commit(bar(C::EMPTY + slot));
          }
          if (!ok) break;
          umma_commit(bar(C::PV_DONE));
          umma_commit(bar(C::EMPTY + slot));
          ++p_i;
          // V(i) to V(i + 1): a K between, but before the last; then the next unit
          v_at += p_i == p_n ? 1 : (p_i + 1 == p_n ? 1 : 2);
          ++tp;
        }
        // every tensor-core operation issued must be complete before TMEM is freed
        umma_commit(bar(C::DRAIN));
      }
      __syncwarp();
      volatile int never = 0;
      mbar_wait(bar(C::DRAIN), 0, &never, p.status, site + C::DRAIN);
    } else {
      if (F8 && warp == kScaleWarp) {
        // ---- 8-bit: the scales of the tiles to come, four keys per lane
        const int site = kRoleRowsQ * 64;
        uint16_t* ring = reinterpret_cast<uint16_t*>(smem + C::OFF_SCALES);
        int t = 0;
        bool ok = true;
        // 32 tiles' scales into L2 (a plain load waits behind the ring's copies in
        // the DRAM queues, several tiles' time)
        auto ahead = [&](const Unit& w, int tile) {
          const long long from = (static_cast<long long>(w.b) * p.H_kv + w.hk) * p.Lk + (tile + lane) * kKeys;
          if (tile + lane < w.t1) {
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.k_scale + from));
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.v_scale + from));
          }
        };
        for (int taken = 0; ok; ++taken) {
          const Unit it = take(taken, site);
          if (it.b < 0) break;
          ahead(it, it.t0);
          const long long row = (static_cast<long long>(it.b) * p.H_kv + it.hk) * p.Lk;
          // (two tiles' loads in flight; one where the registers are few: 35.2 and 37.0 us
          // over 5 x 2 key heads x 56 rows of 256 features, 16 x 96 x 1 of 128 94.6 and 93.3)
          constexpr int BATCH = C::MANY_Q ? 1 : 2;
          for (int x = it.t0; x < it.t1 && ok; x += BATCH) {
            if (((x - it.t0) & 31) == 16) ahead(it, x + 16);
            const int m = min(BATCH, it.t1 - x);
            // (a key past the last takes its scales: nothing uses them)
            uint32_t k4[BATCH][4], v4[BATCH][4];
#pragma unroll
            for (int y = 0; y < BATCH; ++y)
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                const int key = min((x + y) * kKeys + 32 * z + lane, it.end - 1);
                k4[y][z] = __ldg(p.k_scale + row + key);
                v4[y][z] = __ldg(p.v_scale + row + key);
              }
#pragma unroll
            for (int y = 0; y < BATCH; ++y) {
              if (y >= m || !ok) break;
              const int slot = t % kScaleTiles;
              ok = t < kScaleTiles || warp_wait(bar(C::SC_EMPTY + slot), ((t / kScaleTiles) - 1) & 1, abort_flag,
                                                site + C::SC_EMPTY + slot);
              if (!ok) break;
#pragma unroll
              for (int z = 0; z < 4; ++z)
                ring[slot * kKeys + 32 * z + lane] = static_cast<uint16_t>(k4[y][z] | (v4[y][z] << 8));
              warp_arrive(bar(C::SC_FULL + slot), lane);
              ++t;
            }
          }
        }
      } else if (warp < kQWarp + C::Q_THREADS / 32) {
        // ---- the next units' Q, output rows and mask words
        const int site = kRoleRowsQ * 64;
        constexpr int QT = C::Q_THREADS;
        const int qt = tid - 32 * kQWarp;
        int k = 0;  // units with keys
        for (int taken = 0;; ++taken) {
          const Unit it = take(taken, site);
          if (it.b < 0) break;
          if (it.t1 == it.t0) {
            // no key at all: output 0, log-sum-exp -inf
            for (int r = qt >> 3; r < NR; r += QT / 8) {
              int t;
              const int out = out_row(it, r, &t);
              if (out < 0) break;
              uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + static_cast<long long>(out) * p.d);
              for (int x = qt & 7; 8 * x < p.d; x += 8) dst[x] = make_uint4(0, 0, 0, 0);
              if (p.lse && (qt & 7) == 0) p.lse[(it.b * p.H + out % p.H) * p.T + t] = -INFINITY;
            }
            continue;
          }
          const int buf = k & 1;
          if (k > 0) {  // (the softmax threads prepare the first)
            ask_q(it, qt, QT);
            const bool ok = prepare_q(std::integral_constant<int, QT>{}, it, buf, qt, [&]() {
              return k < 2 || warp_wait(bar(C::Q_EMPTY + buf), ((k >> 1) - 1) & 1, abort_flag, site + C::Q_EMPTY + buf);
            });
            if (!ok) break;
            fence_proxy_async_smem();
            warp_arrive(bar(C::Q_FULL + buf), lane);
          }
          ++k;
        }
      }
    }
  } else {
    if constexpr (C::SPLIT_REGS) regs_increase<C::REGS_SOFT>();
    // ---- softmax: thread = key; warpgroup wg has rows r0 .. r0 + RPT - 1
    const int site = kRoleRowsSoftmax * 64;
    constexpr int RPT = C::RPT, GW = C::GW, GROUPS = C::GROUPS;
    const int wg = warp >> 2, r0 = wg * RPT, kt = tid & 127, w4 = warp & 3;
    const uint32_t nbar = 1 + wg;  // this warpgroup's named barrier
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(w4 * 32) << 16);
    bool ok = true;
    auto wait = [&](int id, uint32_t parity) {
      ok = ok && thread_wait(bar(id), parity, abort_flag, site + id);
    };
    if (!balanced(p) && !ordered) {
      // the first unit's Q before the ring's first copies (it is this CTA's own)
      Unit own;
      const int index = static_cast<int>(blockIdx.x), u = index % p.units;
      own.hk = u / blocks;
      own.rb = u - own.hk * blocks;
      own.b = index / p.units % p.B;
      ask_q(own, tid, SOFT);
    }
    if (kt < RPT) row_ref[r0 + kt] = 0.f;
    named_barrier(nbar, 128);
    int k = 0;       // units with keys
    uint32_t t = 0;  // tiles
    for (int taken = 0;; ++taken) {
      const Unit it = take(taken, site);
      if (it.b < 0) break;
      const int n = it.t1 - it.t0;
      if (n == 0) continue;
      const int buf = k & 1;
      const int rows_here = min(NR, n_rows - it.rb * NR) - r0;  // this warpgroup's (may be <= 0)
      const int k_end = it.end;
      float l[RPT];
#pragma unroll
      for (int r = 0; r < RPT; ++r) l[r] = 0.f;
      if (k > 0) {
        wait(C::Q_FULL + buf, q_phase(k));
      } else {
        prepare_q(std::integral_constant<int, SOFT>{}, it, 0, tid, []() { return true; });
        fence_proxy_async_smem();
        warp_arrive(bar(C::Q_FIRST), lane);
        wait(C::Q_FIRST, 0);
      }
      const float* factor = row_factor(buf) + r0;
      float* ref = row_ref + r0;
      float* shift = row_shift + r0;  // (in the epilogue: 1 / sum)
      bool forced = true, seen = false;  // (seen: of row kt)
      for (int i = 0; i < n; ++i, ++t) {
        const int key = (it.t0 + i) * kKeys + kt;
        float kf = 1.f, ev = 0.f, vinv = 1.f;
        if constexpr (F8) {
          const int slot = t % kScaleTiles;
          wait(C::SC_FULL + slot, (t / kScaleTiles) & 1);
          const uint32_t kv = reinterpret_cast<const uint16_t*>(smem + C::OFF_SCALES)[slot * kKeys + kt];
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::SC_EMPTY + slot));
          const uint32_t kb = kv & 255u, vb = min(kv >> 8, 254u);
          kf = __uint_as_float(kb << 23);
          ev = static_cast<float>(static_cast<int>(vb) - 127);
          vinv = __uint_as_float((254u - vb) << 23);
        }
        // Which of this warp's 32 keys each row sees (a tile inside the prefix: all), a
        // row's bits to a lane: the prefix, then the row's mask words up to the last key.
        // A key that no row of the unit sees is hidden.
        constexpr int WINS = (NR + 31) / 32;
        const bool masked = (it.t0 + i + 1) * kKeys > it.n;
        uint32_t win = 0;  // (of row r0 / 32 * 32 + lane)
        bool hidden = false;
        if (masked) {
          const int off = key - lane - it.n, x = off >> 5, left = k_end - (key - lane);
          const uint32_t prefix = off >= 0 ? 0u : (off <= -32 ? ~0u : (1u << -off) - 1);
          const uint32_t here = left >= 32 ? ~0u : (left <= 0 ? 0u : (1u << left) - 1);
          uint32_t any = 0;
#pragma unroll
          for (int a = 0; a < WINS; ++a) {
            uint32_t w[2] = {0, 0};
            if (lane + 32 * a < NR) {
              const uint32_t* words = reinterpret_cast<const uint32_t*>(row_mask(buf) + (lane + 32 * a) * kMaskWords);
              if (x >= 0 && x < 2 * kMaskWords) w[0] = words[x];
              if (x >= -1 && x < 2 * kMaskWords - 1) w[1] = words[x + 1];
            }
            const uint32_t bits = (__funnelshift_r(w[0], w[1], off & 31) | prefix) & here;
            if (a == 0 || wg == a) win = bits;
            any |= bits;
          }
          hidden = !((__reduce_or_sync(0xffffffffu, any) >> lane) & 1);
        }
        wait(C::S_FULL + (t & 1), (t >> 1) & 1);
        tc_fence_after();
        const uint32_t s_at = t_lane + ((t & 1) ? C::TM_S1 : 0u) + r0;
        // the rows' scores of this key (log2 units, v's exponent added) less their
        // references
        float x[RPT];
        {
          // (all columns requested at once, but for 32 rows of two pieces each)
          constexpr int LG = F8 ? 1 : GROUPS;
#pragma unroll
          for (int g0 = 0; g0 < GROUPS; g0 += LG) {
            if (g0 * GW >= rows_here) continue;
            uint32_t c1[LG][GW], c2[F8 ? LG : 1][GW];
#pragma unroll
            for (int g = 0; g < LG; ++g) {
              if ((g0 + g) * GW >= rows_here) continue;
              tmem_ld_cols<GW>(s_at + (g0 + g) * GW, c1[g]);
              if constexpr (F8) tmem_ld_cols<GW>(s_at + NR + (g0 + g) * GW, c2[g]);
            }
            tmem_ld_wait();
#pragma unroll
            for (int gg = 0; gg < LG; ++gg) {
              const int g = g0 + gg;
              if (g * GW >= rows_here) continue;
#pragma unroll
              for (int r = 0; r < GW; r += 4) {
                float* y = x + g * GW + r;
                const float4 m = *reinterpret_cast<const float4*>(ref + g * GW + r);
                const uint32_t* a = c1[gg] + r;
                if constexpr (F8) {
                  const float4 f = *reinterpret_cast<const float4*>(factor + g * GW + r);
                  const uint32_t* c = c2[gg] + r;
                  float b[4], h[4];
                  fma2(b[0], b[1], __uint_as_float(c[0]), __uint_as_float(c[1]), 1.f / 32.f, 1.f / 32.f,
                       __uint_as_float(a[0]), __uint_as_float(a[1]));
                  fma2(b[2], b[3], __uint_as_float(c[2]), __uint_as_float(c[3]), 1.f / 32.f, 1.f / 32.f,
                       __uint_as_float(a[2]), __uint_as_float(a[3]));
                  mul2(h[0], h[1], f.x, f.y, kf, kf);
                  mul2(h[2], h[3], f.z, f.w, kf, kf);
                  fma2(y[0], y[1], b[0], b[1], h[0], h[1], ev - m.x, ev - m.y);
                  fma2(y[2], y[3], b[2], b[3], h[2], h[3], ev - m.z, ev - m.w);
                } else {
                  fma2(y[0], y[1], __uint_as_float(a[0]), __uint_as_float(a[1]), p.scale_log2, p.scale_log2, -m.x,
                       -m.y);
                  fma2(y[2], y[3], __uint_as_float(a[2]), __uint_as_float(a[3]), p.scale_log2, p.scale_log2, -m.z,
                       -m.w);
                }
              }
            }
          }
          if (masked) {
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
              const uint32_t row = __shfl_sync(0xffffffffu, win, (r0 + r) & 31);
              if (!((row >> lane) & 1)) x[r] = -INFINITY;
            }
          }
        }
        bool move = forced;
        if (!forced) {
          float top = -INFINITY;
#pragma unroll
          for (int r = 0; r < RPT; r += 2)
            if (r / GW * GW < rows_here) top = fmax3(top, x[r], x[r + 1]);
          move = any_of_128(nbar, top > C::SLACK + C::LIFT);
        }
        if (move) {
          // move the references to this tile's maxima (always in a unit's first
          // tile, and while a row has seen no key) and rescale
#pragma unroll
          for (int r = 0; r < RPT; ++r) {
            if (r / GW * GW >= rows_here) continue;
            const float m = warp_max(x[r]);
            if (lane == r) red[(r0 + r) * 4 + w4] = m;
          }
          named_barrier(nbar, 128);
          bool unseen = false;
          if (kt < RPT && kt / GW * GW < rows_here) {
            const float4 m4 = *reinterpret_cast<const float4*>(red + (r0 + kt) * 4);
            const float m = fmaxf(fmax3(m4.x, m4.y, m4.z), m4.w);
            // (a row's first key sets its reference, which was 0, up or down)
            const float by = m == -INFINITY ? 0.f : (seen ? fmaxf(m - C::LIFT, 0.f) : m - C::LIFT);
            seen = seen || m > -INFINITY;
            ref[kt] += by;
            shift[kt] = by;
            unseen = !seen && kt < rows_here && row_live(buf)[r0 + kt];
          }
          forced = any_of_128(nbar, unseen);
#pragma unroll
          for (int r = 0; r < RPT; r += 4) {
            if (r / GW * GW >= rows_here) continue;
            const float4 by = *reinterpret_cast<const float4*>(shift + r);
            x[r] -= by.x;
            x[r + 1] -= by.y;
            x[r + 2] -= by.z;
            x[r + 3] -= by.w;
          }
          if (i > 0) {
            // (a row's first key may move its reference down by any amount; its sums and
            // O are 0 then, and a factor above 1 could be infinite: 0 * inf)
#pragma unroll
            for (int r = 0; r < RPT; ++r)
              if (r / GW * GW < rows_here) l[r] *= ex2_approx(fminf(-shift[r], 0.f));
            wait(C::PV_DONE, (t - 1) & 1);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < C::BLKS * C::PP; ++c)
#pragma unroll 1
              for (int g = 0; g < GROUPS; ++g) {
                if (g * GW >= rows_here) continue;
                const uint32_t o_at =
                    t_lane + C::TM_O + (c / C::PP) * C::NP + (c % C::PP) * NR + r0 + g * GW;
                uint32_t o[GW];
                tmem_ld_cols<GW>(o_at, o);
                tmem_ld_wait();
#pragma unroll
                for (int r = 0; r < GW; ++r)
                  o[r] = __float_as_uint(__uint_as_float(o[r]) * ex2_approx(fminf(-shift[g * GW + r], 0.f)));
                tmem_st_cols<GW>(o_at, o);
              }
            tmem_st_wait();
          }
        }
        tc_fence_before();
        // weights; the product before must have read P (a second buffer of P measured
        // nothing: this wait is over long before the weights are ready)
        if (t > 0) wait(C::PV_DONE, (t - 1) & 1);
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
          if (g * GW >= rows_here) continue;
          uint32_t w1[GW / 2], w2[GW / 2], w3[GW / 4];  // (8-bit: the first GW / 4 of each)
#pragma unroll
          for (int r = 0; r < GW; r += 2) {
            const int a = g * GW + r;
            const float p0 = ex2_approx(x[a]), p1 = ex2_approx(x[a + 1]);
            if constexpr (F8) {
              fma2(l[a], l[a + 1], p0, p1, vinv, vinv, l[a], l[a + 1]);
              const uint32_t h = pack_half2(p0, p1);
              const uint32_t b1 = half2_to_e5m2x2(h);
              const uint32_t h2 = half2_sub(h, e5m2x2_to_half2(b1));
              const uint32_t b2 = half2_to_e5m2x2(h2);
              const uint32_t b3 = half2_to_e5m2x2(half2_sub(h2, e5m2x2_to_half2(b2)));
              const int x4 = r >> 2;
              if ((r & 2) == 0) {
                w1[x4] = b1;
                w2[x4] = b2;
                w3[x4] = b3;
              } else {
                w1[x4] |= b1 << 16;
                w2[x4] |= b2 << 16;
                w3[x4] |= b3 << 16;
              }
            } else {
              add2(l[a], l[a + 1], l[a], l[a + 1], p0, p1);
              // the first piece is cut, not rounded: its bits are p's own
              const uint32_t u0 = __float_as_uint(p0) & 0xffff0000u, u1 = __float_as_uint(p1) & 0xffff0000u;
              w1[r >> 1] = __byte_perm(u0, u1, 0x7632);
              w2[r >> 1] = pack_bf16x2(p0 - __uint_as_float(u0), p1 - __uint_as_float(u1));
            }
          }
          // 16-byte units [column of units][key]: 16 (8-bit) or 8 rows of a piece
          constexpr int COL = kKeys * 16;
          if constexpr (F8 && NR == 4) {
            // the three pieces in one unit
            st_shared_v4(sP + kt * 16, w1[0], w2[0], w3[0], 0);
          } else if constexpr (F8 && NR == 8) {
            // two pieces to a unit; nothing reads the second half of the last
            const uint32_t to = sP + kt * 16;
            st_shared_v4(to, w1[0], w1[1], w2[0], w2[1]);
            st_shared_v4(to + COL, w3[0], w3[1], 0, 0);
          } else if constexpr (F8 && GW == 8) {
            // half a unit
            const uint32_t to = sP + r0 / 16 * COL + kt * 16 + (r0 & 8);
            st_shared_v2(to, w1[0], w1[1]);
            st_shared_v2(to + (NR / 16) * COL, w2[0], w2[1]);
            st_shared_v2(to + 2 * (NR / 16) * COL, w3[0], w3[1]);
          } else if constexpr (F8) {
            const uint32_t to = sP + (r0 / 16 + g) * COL + kt * 16;
            st_shared_v4(to, w1[0], w1[1], w1[2], w1[3]);
            st_shared_v4(to + (NR / 16) * COL, w2[0], w2[1], w2[2], w2[3]);
            st_shared_v4(to + 2 * (NR / 16) * COL, w3[0], w3[1], w3[2], w3[3]);
          } else {
#pragma unroll
            for (int h = 0; h < GW / 8; ++h) {
              const uint32_t to = sP + ((r0 + g * GW) / 8 + h) * COL + kt * 16;
              st_shared_v4(to, w1[4 * h], w1[4 * h + 1], w1[4 * h + 2], w1[4 * h + 3]);
              st_shared_v4(to + (NR / 8) * COL, w2[4 * h], w2[4 * h + 1], w2[4 * h + 2], w2[4 * h + 3]);
            }
          }
        }
        if (wg == 0 && masked && __any_sync(0xffffffffu, hidden)) {
          // a hidden key's V may hold anything, and 0 * NaN would be NaN (the ring has
          // K(0) K(1) V(0) K(2) ... V(last) of a unit)
          const int before = 2 * static_cast<int>(t) + (i + 1 < n ? 2 : 1);
          for (int blk = 0; blk < blks; ++blk) {
            const int item = before * blks + blk, sl = item % C::SLOTS;
            wait(C::FULL + sl, (item / C::SLOTS) & 1);
            if (hidden) {
#pragma unroll 1
              for (int c = 0; c < C::SLOT / C::CHUNK; ++c)
#pragma unroll 1
                for (int u = 0; u < 8; ++u)
                  st_shared_v4(s_base + sl * C::SLOT + c * C::CHUNK + kt * 128 + u * 16, 0, 0, 0, 0);
            }
          }
        }
        fence_proxy_async_smem();
        warp_arrive(bar(C::P_FULL), lane);
      }

      // ---- epilogue: sums over the keys, then O
      {
        // (the lanes of a row's group all hold its sum)
        const float y = warp_sums<RPT>(l, lane);
        if (lane % (32 / RPT) == 0) red[(r0 + lane / (32 / RPT)) * 4 + w4] = y;
      }
      wait(C::PV_DONE, (t - 1) & 1);
      tc_fence_after();
      const bool good = ok && *abort_flag == 0;
      named_barrier(nbar, 128);
      const bool whole = it.splits == 1;
      const int* outs = row_out(buf) + r0;
      const long long part = static_cast<long long>(it.part - it.b) * p.T * p.H;  // (rows count from sequence 0)
      if (kt < rows_here && kt < RPT) {
        const float4 l4 = *reinterpret_cast<const float4*>(red + (r0 + kt) * 4);
        float L = l4.x + l4.y + l4.z + l4.w;
        float m = ref[kt];
        if (!row_live(buf)[r0 + kt] || !good) {  // an empty row (or a CTA that gave up)
          L = 0.f;
          m = -INFINITY;
        }
        shift[kt] = L > 0.f ? (whole ? 1.f / L : 1.f) : 0.f;
        if (!whole) {
          p.part_m[part + outs[kt]] = L > 0.f ? m : -INFINITY;
          p.part_l[part + outs[kt]] = L;
        } else if (p.lse) {
          p.lse[row_lse(buf)[r0 + kt]] = L > 0.f ? (m + __log2f(L)) * 0.69314718055994531f : -INFINITY;
        }
      }
      if (kt < RPT) ref[kt] = 0.f;  // (for the next unit)
      named_barrier(nbar, 128);
      const int f0 = C::M_O == 64 ? w4 * 16 + lane : kt;
      const bool holds = C::M_O == 128 || lane < 16;
      // (eight rows at a time and no unrolling past that: this runs once per unit)
#pragma unroll 1
      for (int blk = 0; blk < blks; ++blk) {
        const int f = blk * 128 + f0;
        const bool stores = holds && f < p.d;
#pragma unroll 1
        for (int g = 0; g < rows_here; g += 8) {
          if (g >= RPT) break;
          uint32_t y[C::PP][8];
#pragma unroll
          for (int piece = 0; piece < C::PP; ++piece)
            tmem_ld_cols<8>(t_lane + C::TM_O + blk * C::NP + piece * NR + r0 + g, y[piece]);
          tmem_ld_wait();
          if (!stores) continue;
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            if (g + r >= rows_here) break;
            float o = __uint_as_float(y[C::PP - 1][r]);
#pragma unroll
            for (int piece = C::PP - 2; piece >= 0; --piece) o += __uint_as_float(y[piece][r]);
            const float a = shift[g + r];
            const long long row = outs[g + r];
            if (whole)
              static_cast<__nv_bfloat16*>(p.out)[row * p.d + f] = __float2bfloat16_rn(a > 0.f ? o * a : 0.f);
            else
              p.part_o[(part + row) * W + f] = a > 0.f ? o : 0.f;
          }
        }
      }
      tc_fence_before();
      warp_arrive(bar(C::O_FREE), lane);
      warp_arrive(bar(C::Q_EMPTY + buf), lane);
      ++k;
    }
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
  if (tid == 0 && *abort_flag != 0 && atomicCAS(&p.status->code, 0, 7 /* MHA_ERR_TIMEOUT */) == 0) {
    p.status->site = *abort_flag - 1;
    p.status->block = static_cast<int>(blockIdx.x);
  }
}

// Merges a row's partials:
//   o = sum_x 2^(m_x - M) o_x / sum_x 2^(m_x - M) l_x,  M = max_x m_x
// over the splits x of its sequence.  A row has WARPS warps of an eight-warp block,
// which divide its partials (eight when one long
// sequence is spread over the machine, one when there are few splits and many rows); a lane holds W / 32 neighbouring
// features, and a warp's first four o_x are requested together with the m_x.
template <int W, int WARPS>
__global__ void __launch_bounds__(256) rows_combine_kernel(const __grid_constant__ RowsParams p) {
  constexpr int EPL = W / 32, AHEAD = 4;
  __shared__ float sums[8][WARPS > 1 ? W + 1 : 1];
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int part = warp % WARPS;
  const long long rows = static_cast<long long>(p.B) * p.T * p.H;
  const long long row = static_cast<long long>(blockIdx.x) * (8 / WARPS) + warp / WARPS;
  const int bt = static_cast<int>(row / p.H), h = static_cast<int>(row - static_cast<long long>(bt) * p.H);
  const int b = bt / p.T;
  // The lengths may be read before the wait: the rows kernel, which does not write
  // them, let this one start after its own wait for whatever came before.
  int splits = 1;
  long long at = row, step = rows;  // the first partial; from one to the next
  if (row < rows) {
    if (balanced(p)) {
      int first, per;
      balance(p, lane, &first, &splits, &per);
      splits = __shfl_sync(0xffffffffu, splits, b);
      step = static_cast<long long>(p.T) * p.H;
      at += (__shfl_sync(0xffffffffu, first, b) - b) * step;
    } else {
      splits = unit_of(p, 0, 1, b, 0, 0).splits;
    }
  }
  griddep_wait();  // the splits' partials are complete and visible
  float o[EPL], L = 0.f, M = -INFINITY;
#pragma unroll
  for (int e = 0; e < EPL; ++e) o[e] = 0.f;
  if (splits > 1) {
    auto load = [&](int x, float (&y)[EPL]) {
      const float* src = p.part_o + (at + x * step) * W + lane * EPL;
      if constexpr (EPL == 2) {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
        y[0] = v.x, y[1] = v.y;
      } else {
#pragma unroll
        for (int e = 0; e < EPL; e += 4) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(src + e));
          y[e] = v.x, y[e + 1] = v.y, y[e + 2] = v.z, y[e + 3] = v.w;
        }
      }
    };
    float first[AHEAD][EPL], m[2], a[2];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (part + i * WARPS < splits) load(part + i * WARPS, first[i]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // (kMaxRowSplits = 64)
      const int x = lane + 32 * i;
      m[i] = -INFINITY;
      a[i] = 0.f;
      if (x < splits) {
        m[i] = __ldcg(p.part_m + at + x * step);
        a[i] = __ldcg(p.part_l + at + x * step);
      }
    }
    M = warp_max(fmaxf(m[0], m[1]));
    if (M != -INFINITY) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float f = ex2_approx(m[i] - M);  // 0 for a split the row sees nothing of
        L = fmaf(f, a[i], L);
        a[i] = f;
      }
#pragma unroll
      for (int i = 16; i > 0; i >>= 1) L += __shfl_xor_sync(0xffffffffu, L, i);
      auto add = [&](int x, const float (&y)[EPL]) {
        const float f = __shfl_sync(0xffffffffu, x < 32 ? a[0] : a[1], x & 31);
#pragma unroll
        for (int e = 0; e < EPL; ++e) o[e] = fmaf(f, y[e], o[e]);
      };
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (part + i * WARPS < splits) add(part + i * WARPS, first[i]);
#pragma unroll 4
      for (int x = part + AHEAD * WARPS; x < splits; x += WARPS) {
        float y[EPL];
        load(x, y);
        add(x, y);
      }
    }
  }
  if constexpr (WARPS > 1) {
    if (part != 0) {
#pragma unroll
      for (int e = 0; e < EPL; ++e) sums[warp][lane + 32 * e] = o[e];
    }
    __syncthreads();
    if (part == 0) {
#pragma unroll
      for (int x = 1; x < WARPS; ++x)
#pragma unroll
        for (int e = 0; e < EPL; ++e) o[e] += sums[warp + x][lane + 32 * e];
    }
  }
  if (part != 0 || splits <= 1) return;  // (a single split wrote the row itself)
  const float inv = L > 0.f ? 1.f / L : 0.f;
  uint32_t out[EPL / 2];
#pragma unroll
  for (int e = 0; e < EPL; e += 2) out[e / 2] = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
  // (d is a multiple of 8: a lane's features are all inside it or all past it)
  if (lane * EPL < p.d) {
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + row * p.d + lane * EPL);
    if constexpr (EPL == 2) *dst = out[0];
    else if constexpr (EPL == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
    else *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
  }
  if (p.lse && lane == 0)
    p.lse[(static_cast<long long>(b) * p.H + h) * p.T + (bt - b * p.T)] =
        L > 0.f ? (M + __log2f(L)) * 0.69314718055994531f : -INFINITY;
}

template <bool F8, int W, int NR>
cudaError_t launch_rows_cfg(const RowsParams& p, cudaStream_t stream, LaunchInfo* info) {
  using C = RowsCfg<F8, W, NR>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static bool attr_set[64] = {};
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(rows_kernel<F8, W, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  // one CTA per unit; running CTAs take over the units of those not started
  const dim3 grid(static_cast<unsigned>(p.B * p.units * p.n_splits));
  e = launch_serialized(rows_kernel<F8, W, NR>, grid, dim3(C::THREADS), C::SMEM, stream, p);
  if (e != cudaSuccess) return e;
  if (info) {
    info->kernels = 1;
    info->grid = static_cast<int>(grid.x);
    info->block = C::THREADS;
    info->smem = C::SMEM;
  }
  return e;
}

// Calls f with the kernel's configuration for R rows per key head of d features.  Rows
// beyond R cost their weights all the same (8 bits, 128 features: one row over 16 x 96
// heads x 1,024 to 2,048 keys 94.5 us in units of four and 95.4 of eight, four over 2 x
// 8 x 40k to 65k 42.2 and 43.2; bf16, 64 features: four over 128 x 8 heads x 250 keys 25
// us in units of eight and 27 of sixteen; wider heads, one CTA per SM, the same in both).
template <typename F>
void with_config(bool f8, int d, int R, F&& f) {
  if (f8 && d <= 128) {
    if (R <= 4) f(RowsCfg<true, 128, 4>{});
    else if (R <= 8) f(RowsCfg<true, 128, 8>{});
    else if (R <= 16) f(RowsCfg<true, 128, 16>{});
    else if (R <= 32) f(RowsCfg<true, 128, 32>{});
    else f(RowsCfg<true, 128, 64>{});
  } else if (f8) {
    if (R <= 4) f(RowsCfg<true, 256, 4>{});
    else if (R <= 8) f(RowsCfg<true, 256, 8>{});
    else if (R <= 16) f(RowsCfg<true, 256, 16>{});
    else f(RowsCfg<true, 256, 32>{});
  } else if (d <= 64) {
    if (R <= 8) f(RowsCfg<false, 64, 8>{});
    else if (R <= 16) f(RowsCfg<false, 64, 16>{});
    else if (R <= 32) f(RowsCfg<false, 64, 32>{});
    else f(RowsCfg<false, 64, 64>{});
  } else if (d <= 128) {
    if (R <= 16) f(RowsCfg<false, 128, 16>{});
    else if (R <= 32) f(RowsCfg<false, 128, 32>{});
    else f(RowsCfg<false, 128, 64>{});
  } else {
    if (R <= 16) f(RowsCfg<false, 256, 16>{});
    else f(RowsCfg<false, 256, 32>{});
  }
}

// The kernel for T rows of G query heads per key head.
//   More than 64 rows over a bf16 cache: along M (3 x 8 key heads x 16,000 keys of
//   128 features: 60 rows 56 us along N and 58 along M, 96 rows 68 and 58, 128 rows
//   68 and 60; 64 rows of 8 blocks: 566 and 269 at 2,048 rows x 32,000 keys).
//   A row or two over a short 8-bit cache: the CUDA cores.  us there and on the tensor
//   cores, calls of a graph that read from DRAM, features x keys of full caches:
//     128 x 8 heads   64 x 64  5.7 and 16.1    64 x 256 10.8 and 17.0 (16 to 256 keys
//                     9.2 and 17.6)            64 x 512 17.3 and 21.2
//     16 x 96 heads   128 x 128 16.5 and 19.4  128 x 256 28.3 and 22.4
//     16 x 8 heads    64 x 256 7.2 and 6.1
//     1 x 8 heads     64 x 128 3.2 and 4.6     64 x 256 4.6 and 5.0
//     32 x 4 heads    256 x 64 6.4 and 7.0
//     128 x 8 key heads of two rows            64 x 128 11.1 and 14.6
//   One border for any width and number of heads (keys x features x rows): narrow heads
//   just past it would gain 4 us here, a hundred heads at its end 1 us there.
RowsForm rows_form(bool f8, int d, int T, int G, int Lk) {
  if (!f8 && d <= 128 && T * G > 64) return kRowsBlock;
  if (f8 && T == 1 && G <= kShortRows && static_cast<long long>(Lk) * d * G <= kShortWork) return kRowsShort;
  return kRowsKeys;
}

template <int W>
cudaError_t launch_combine(const RowsParams& p, cudaStream_t stream) {
  const long long rows = static_cast<long long>(p.B) * p.T * p.H;
  const bool many = p.n_splits >= 8;
  const int per_block = many ? 1 : 8;
  return launch_serialized(many ? rows_combine_kernel<W, 8> : rows_combine_kernel<W, 1>,
                           dim3(static_cast<unsigned>((rows + per_block - 1) / per_block)), dim3(256), 0, stream, p);
}

}  // namespace

RowsPlan rows_plan(int B, int T, int H, int H_kv, int Lk, int d, bool f8) {
  const int R = T * (H / H_kv);
  RowsPlan plan = {};
  plan.form = rows_form(f8, d, T, H / H_kv, Lk);
  if (plan.form == kRowsShort) {
    plan.units = H_kv;
    plan.splits = 1;
    return plan;
  }
  int rows = kBlockRows, ctas = 1;  // rows per unit, CTAs per SM
  plan.width = d <= 64 ? 64 : 128;
  if (plan.form == kRowsKeys)
    with_config(f8, d, R, [&](auto cfg) {
      using C = decltype(cfg);
      plan.width = C::W;
      rows = C::NR;
      ctas = C::MIN_BLOCKS;
    });
  plan.units = static_cast<long long>(H_kv) * ((R + rows - 1) / rows);
  const long long base = plan.units * B;
  const long long slots = static_cast<long long>(kSms) * ctas;
  const long long tiles = (Lk + kKeys - 1) / kKeys;
  // Time in half tiles, sequences counted at the cache's capacity: a unit costs
  // its tiles and five more (its Q, first tile and epilogue); with several units
  // to a CTA the last ones end half a unit apart; partials cost a second kernel
  // (some four tiles) and are written and read at about the rate of the keys.
  // (3 sequences x 8 key heads x 4 blocks of 64 rows x 16,411 keys of 128 features,
  // by splits: 1 141 us, 2 118, 3 105, 5 113, 7 115; 5 x 2 x 2 blocks of 32 rows x
  // 20,011 keys of 256 features in 8 bits: 4 67 us, 6 52, 7 48, 8 49, 14 51.)
  long long best = -1;
  for (long long S = 1; S <= kMaxRowSplits && S <= tiles && (S == 1 || base * (S - 1) < 4 * slots); ++S) {
    const long long per = 2 * ((tiles + S - 1) / S) + 10;
    const long long units = base * S;
    const long long merge = S == 1 ? 0 : 8 + units * rows / (slots * (f8 ? 16 : 32));
    const long long cost = (units <= slots ? per : units * per / slots + per / 2) + merge;
    if (best >= 0 && cost >= best) continue;
    best = cost;
    plan.splits = static_cast<int>(S);
  }
  plan.part_rows = plan.splits > 1 ? static_cast<size_t>(plan.splits) * B * T * H : 0;
  return plan;
}

int rows_tile_keys() { return kKeys; }
int rows_box_keys() { return kBoxKeys; }

cudaError_t launch_rows(const RowsParams& p, cudaStream_t stream, LaunchInfo* info) {
  const bool f8 = p.k_scale != nullptr;
  const int R = p.T * p.G;
  cudaError_t e = cudaSuccess;
  if (p.form == kRowsShort) {
    e = launch_rows_short(p, stream, info);
  } else if (p.form == kRowsBlock) {
    e = launch_rows_block(p, stream, info);
  } else {
    with_config(f8, p.d, R, [&](auto cfg) {
      using C = decltype(cfg);
      e = launch_rows_cfg<C::F8, C::W, C::NR>(p, stream, info);
    });
  }
  if (e != cudaSuccess || p.n_splits == 1) return e;
  if (info) info->kernels = 2;
  if (!f8 && p.d <= 64) return launch_combine<64>(p, stream);
  return p.d <= 128 ? launch_combine<128>(p, stream) : launch_combine<256>(p, stream);
}

}  // namespace mha

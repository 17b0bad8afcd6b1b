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
// bf16 cache: kind::f16, q exact, p as two bf16 pieces (2^-16).
//
// Online softmax (scores in log2 units, q's factor scale * log2 e): the
// reference m of a row moves only when a tile's largest score exceeds it by
// more than a slack (8, or 5 for the 8-bit pieces' range); then O (in TMEM)
// and the sums are rescaled.  Sums are float32, one partial per thread and row,
// added up once at the end.
//
// The key axis is split over gridDim.y CTAs per (sequence, key head, block of
// rows) when those alone would leave SMs idle; each sequence's own key count is
// divided, so short sequences of a ragged batch use fewer splits.  Partials
// (o, m, l) go to the workspace and rows_combine_kernel merges them exactly.
//
// 192 threads: warps 0-3 softmax and epilogue (thread = key = TMEM lane), warp
// 4 TMEM allocation and MMA issue, warp 5 TMA producer.  The MMA warp runs
// S(0), S(1), PV(0), S(2), PV(1), ...: the next tile's scores are computed
// while the softmax works on this one's.  K and V tiles share one ring in that
// order.  Every wait is bounded (abort flag, MHA_ERR_TIMEOUT).
#include <cuda_bf16.h>

#include "fp8.cuh"
#include "kernels.h"

namespace mha {
namespace {

constexpr int kKeys = 128;         // keys per tile
constexpr int kBoxKeys = 32;       // keys per TMA box: a ragged last tile loads only what it needs
constexpr int kRowThreads = 192;
constexpr int kMmaWarp = 4, kLoadWarp = 5;
constexpr int kRoleRowsLoad = 16, kRoleRowsMma = 17, kRoleRowsSoftmax = 18;

template <bool F8_, int W_, int NR_>
struct RowsCfg {
  static constexpr bool F8 = F8_;
  static constexpr int W = W_;    // widest head
  static constexpr int NR = NR_;  // rows per CTA
  static constexpr int EB = F8 ? 1 : 2;                  // bytes per cached element
  static constexpr int CHUNK = kKeys * 128;              // [128 keys x 128 B], 128-byte swizzle
  static constexpr int TILE = kKeys * W * EB;            // a K or V tile
  static constexpr int QP = F8 ? 2 : 1;                  // pieces of q
  static constexpr int PP = F8 ? 3 : 2;                  // pieces of p
  static constexpr int NQ = QP * NR, NP = PP * NR;       // columns of S^T and O^T
  static constexpr int Q_BYTES = NQ * W * EB;
  static constexpr int P_BYTES = kKeys * NP * EB;
  static constexpr int MISC = NR > 32 ? 4096 : 2048;
  // two CTAs per SM when three tiles of the ring fit, else one with a deep ring
  static constexpr int FIXED = Q_BYTES + P_BYTES + MISC + 1024;
  static constexpr int SLOTS2 = (115712 - FIXED) / TILE;
  static constexpr bool TWO = SLOTS2 >= 3 && NR <= 32;
  static constexpr int SLOTS = TWO ? SLOTS2 : (232448 - FIXED) / TILE;
  static constexpr int MIN_BLOCKS = TWO ? 2 : 1;
  static_assert(SLOTS >= 3, "ring");
  static constexpr int OFF_Q = SLOTS * TILE;
  static constexpr int OFF_P = OFF_Q + Q_BYTES;
  static constexpr int OFF_MISC = OFF_P + P_BYTES;
  static constexpr int SMEM = OFF_MISC + MISC + 1024;
  // barriers
  static constexpr int FULL = 0;              // + slot
  static constexpr int EMPTY = SLOTS;         // + slot
  static constexpr int Q_FULL = 2 * SLOTS;    // 128 arrivals
  static constexpr int S_FULL = Q_FULL + 1;   // + buffer
  static constexpr int P_FULL = S_FULL + 2;   // 128 arrivals
  static constexpr int PV_DONE = P_FULL + 1;
  static constexpr int DRAIN = PV_DONE + 1;
  static constexpr int NBAR = DRAIN + 1;
  // misc area: barriers, TMEM slot, abort flag, then per-row values
  static constexpr int OFF_TMEM = OFF_MISC + 8 * NBAR;
  static constexpr int OFF_ABORT = OFF_TMEM + 4;
  static constexpr int OFF_ROWS = OFF_MISC + (8 * NBAR + 8 + 15) / 16 * 16;
  // [factor | reference | alpha | red: 4 warps | output row | draft], NR each
  static_assert(OFF_ROWS - OFF_MISC + 9 * NR * 4 <= MISC, "misc area");
  // TMEM: S0 | S1 | O (per 128 features)
  static constexpr int M_O = W == 64 ? 64 : 128;         // rows of the O^T tile
  static constexpr int BLKS = W <= 128 ? 1 : 2;          // blocks of 128 features
  static constexpr uint32_t TM_S1 = NQ, TM_O = 2 * NQ;
  static constexpr uint32_t TM_USED = 2 * NQ + BLKS * NP;
  static constexpr uint32_t TMEM_COLS =
      TM_USED <= 32 ? 32 : (TM_USED <= 64 ? 64 : (TM_USED <= 128 ? 128 : (TM_USED <= 256 ? 256 : 512)));
  static_assert(TM_USED <= 512 && (!TWO || TMEM_COLS <= 256), "TMEM budget");
  static_assert(OFF_Q % 1024 == 0 && OFF_P % 128 == 0 && OFF_MISC % 16 == 0, "alignment");
  static constexpr float SLACK = F8 ? 5.f : 8.f;         // reference moves beyond this (log2)
  static constexpr float LIFT = F8 ? 10.f : 0.f;         // weights are 2^LIFT at the reference
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

// True for every softmax thread when any of them passes true (named barrier 1).
__device__ __forceinline__ bool any_of_128(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x))
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

// What a CTA works on.
struct RowsWork {
  int n;              // prefix keys
  int live;           // drafted tokens (rows) of the sequence
  int end;            // keys any row may see
  int per, active;    // tiles per split, splits with work (>= 1)
};
__device__ __forceinline__ RowsWork rows_work(const RowsParams& p, int b) {
  RowsWork w;
  const int n = __ldg(p.prefix_lens + b);
  w.n = n < 0 ? 0 : (n > p.Lk ? p.Lk : n);
  w.live = p.T;
  if (p.draft_lens) {
    const int live = __ldg(p.draft_lens + b);
    w.live = live < 0 ? 0 : (live > p.T ? p.T : live);
  }
  w.end = p.drafts ? min(p.Lk, w.n + w.live) : w.n;
  if (w.live == 0) w.end = 0;  // every row is empty
  const int tiles = (w.end + kKeys - 1) / kKeys;
  w.per = (tiles + p.n_splits - 1) / p.n_splits;
  w.active = w.per > 0 ? (tiles + w.per - 1) / w.per : 1;
  return w;
}

template <bool F8, int W, int NR>
__global__ void __launch_bounds__(kRowThreads, (RowsCfg<F8, W, NR>::MIN_BLOCKS))
    rows_kernel(const __grid_constant__ RowsParams p) {
  using C = RowsCfg<F8, W, NR>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t s_base = smem_u32(smem);
  auto bar = [&](int id) { return s_base + C::OFF_MISC + 8u * static_cast<uint32_t>(id); };
  const uint32_t sQ = s_base + C::OFF_Q, sP = s_base + C::OFF_P;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_TMEM);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
  float* row_factor = reinterpret_cast<float*>(smem + C::OFF_ROWS);
  float* row_ref = row_factor + NR;
  float* row_alpha = row_ref + NR;
  float* red = row_alpha + NR;                       // [4][NR]
  int* row_out = reinterpret_cast<int*>(red + 4 * NR);  // output row, -1: none
  int* row_t = row_out + NR;                         // drafted token, -1: an empty row
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int tid = static_cast<int>(threadIdx.x);

  // (rows block fastest, then key head: CTAs that read the same or neighbouring
  // cache rows run together)
  const int n_rows = p.T * p.G;
  const int blocks = (n_rows + NR - 1) / NR;
  int x = static_cast<int>(blockIdx.x);
  const int rb = x % blocks;
  x /= blocks;
  const int hk = x % p.H_kv, b = x / p.H_kv;
  const int split = static_cast<int>(blockIdx.y);
  const int rows_here = min(NR, n_rows - rb * NR);

  if (tid == 0) {
    for (int s = 0; s < C::SLOTS; ++s) {
      mbar_init(bar(C::FULL + s), 1);
      mbar_init(bar(C::EMPTY + s), 1);
    }
    mbar_init(bar(C::Q_FULL), 128);
    mbar_init(bar(C::S_FULL), 1);
    mbar_init(bar(C::S_FULL + 1), 1);
    mbar_init(bar(C::P_FULL), 128);
    mbar_init(bar(C::PV_DONE), 1);
    mbar_init(bar(C::DRAIN), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), C::TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == kLoadWarp && lane == 0) {
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();  // global memory only from here on

  const RowsWork w = rows_work(p, b);
  const int k_begin = split * w.per * kKeys;
  const int k_end = min(w.end, k_begin + w.per * kKeys);
  const int n = (k_end > k_begin) ? (k_end - k_begin + kKeys - 1) / kKeys : 0;
  const bool works = split < w.active;
  // order of the ring: K0 K1 V0 K2 V1 ... V(n-1)
  auto k_item = [&](int i) { return i == 0 ? 0 : 2 * i - 1; };
  auto v_item = [&](int i) { return i == n - 1 ? 2 * n - 1 : 2 * i + 2; };

  if (warp == kLoadWarp) {
    // ---- TMA producer
    const int site = kRoleRowsLoad * 64;
    const int chunks = (p.d * C::EB + 127) / 128;
    int item = 0;
    bool ok = true;
    auto load = [&](const CUtensorMap* map, int tile) {
      const int s = item % C::SLOTS;
      if (item >= C::SLOTS &&
          !mbar_wait(bar(C::EMPTY + s), ((item / C::SLOTS) - 1) & 1, abort_flag, p.status,
                     site + C::EMPTY + s))
        return false;
      if (elect_one()) {
        const int key = k_begin + tile * kKeys;
        const int boxes = (min(kKeys, k_end - key) + kBoxKeys - 1) / kBoxKeys;
        mbar_arrive_expect_tx(bar(C::FULL + s), static_cast<uint32_t>(boxes * chunks * kBoxKeys * 128));
        for (int c = 0; c < chunks; ++c)
          for (int x = 0; x < boxes; ++x)
            tma_load_4d(s_base + s * C::TILE + c * C::CHUNK + x * kBoxKeys * 128, map,
                        bar(C::FULL + s), c * (128 / C::EB), hk, key + x * kBoxKeys, b);
      }
      __syncwarp();
      ++item;
      return true;
    };
    if (n > 0) ok = load(&p.tm_k, 0);
    for (int i = 0; i < n && ok; ++i) {
      if (i + 1 < n) ok = load(&p.tm_k, i + 1);
      if (ok) ok = load(&p.tm_v, i);
    }
    // every copy started must land before the CTA exits
    volatile int never = 0;
    for (int t = (item > C::SLOTS ? item - C::SLOTS : 0); t < item; ++t)
      mbar_wait(bar(C::FULL + t % C::SLOTS), (t / C::SLOTS) & 1, &never, p.status, site + C::FULL);
  } else if (warp == kMmaWarp) {
    // ---- MMA issuer
    const int site = kRoleRowsMma * 64;
    constexpr int KSTEP = F8 ? 32 : 16;                 // reduction elements per MMA
    const int n_ks = (p.d + KSTEP - 1) / KSTEP;
    constexpr uint32_t idesc_s = F8 ? idesc_f8_f32(128, C::NQ, 0, false, false)
                                    : idesc_bf16_f32(128, C::NQ, false, false);
    constexpr uint32_t idesc_o = F8 ? idesc_f8_f32(C::M_O, C::NP, 1, true, true)
                                    : idesc_bf16_f32(C::M_O, C::NP, true, true);
    // K: rows of 128 bytes per chunk, 8-row groups 1024 B apart, +32 B per step
    // inside a chunk.  V transposed: features contiguous in a 128-byte row, next
    // chunk of features CHUNK apart, 8-key groups 1024 B apart.
    const uint64_t dk0 = smem_desc_sw128(s_base, 16, 1024);
    const uint64_t dv0 = smem_desc_sw128(s_base, C::CHUNK, 1024);
    const uint64_t dq0 = smem_desc_plain(sQ, C::NQ * 16, 128);
    const uint64_t dp0 = smem_desc_plain(sP, 128, kKeys * 16);
    const int blks = W <= 128 ? 1 : (p.d + 127) / 128;
    auto issue_s = [&](int i) {
      const int it = k_item(i), s = it % C::SLOTS;
      if (!mbar_wait(bar(C::FULL + s), (it / C::SLOTS) & 1, abort_flag, p.status, site + C::FULL + s))
        return false;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t d = tmem + ((i & 1) ? C::TM_S1 : 0u);
        const uint64_t a = dk0 + static_cast<uint64_t>((s * C::TILE) >> 4);
        for (int ks = 0; ks < n_ks; ++ks)
          umma<F8>(d, a + static_cast<uint64_t>(((ks >> 2) * C::CHUNK + (ks & 3) * 32) >> 4),
                   dq0 + static_cast<uint64_t>(ks * 2 * C::NQ), idesc_s, ks > 0 ? 1u : 0u);
        umma_commit(bar(C::S_FULL + (i & 1)));
        umma_commit(bar(C::EMPTY + s));
      }
      __syncwarp();
      return true;
    };
    bool ok = n > 0 && mbar_wait(bar(C::Q_FULL), 0, abort_flag, p.status, site + C::Q_FULL) && issue_s(0);
    for (int i = 0; i < n && ok; ++i) {
      if (i + 1 < n && !(ok = issue_s(i + 1))) break;
      const int it = v_item(i), s = it % C::SLOTS;
      ok = mbar_wait(bar(C::FULL + s), (it / C::SLOTS) & 1, abort_flag, p.status, site + C::FULL + s) &&
           mbar_wait(bar(C::P_FULL), i & 1, abort_flag, p.status, site + C::P_FULL);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        for (int blk = 0; blk < blks; ++blk) {
          const uint32_t d = tmem + C::TM_O + blk * C::NP;
          const uint64_t a =
              dv0 + static_cast<uint64_t>((s * C::TILE + blk * (F8 ? 1 : 2) * C::CHUNK) >> 4);
#pragma unroll
          for (int ks = 0; ks < kKeys / KSTEP; ++ks)
            umma<F8>(d, a + static_cast<uint64_t>((ks * KSTEP * 128) >> 4),
                     dp0 + static_cast<uint64_t>((ks * KSTEP * 16) >> 4), idesc_o,
                     (i > 0 || ks > 0) ? 1u : 0u);
        }
        umma_commit(bar(C::PV_DONE));
        umma_commit(bar(C::EMPTY + s));
      }
      __syncwarp();
    }
    // every tensor-core operation issued must be complete before TMEM is freed
    if (elect_one()) umma_commit(bar(C::DRAIN));
    __syncwarp();
    volatile int never = 0;
    mbar_wait(bar(C::DRAIN), 0, &never, p.status, site + C::DRAIN);
  } else if (works) {
    // ---- softmax: thread = key
    const int site = kRoleRowsSoftmax * 64;
    // per-row values (row r of the block: drafted token and query head)
    if (tid < NR) {
      int out = -1, t = -1;
      if (tid < rows_here) {
        const int gr = rb * NR + tid;
        t = gr / p.G;
        out = (b * p.T + t) * p.H + hk * p.G + gr % p.G;
        if (t >= w.live) t = -1;
      }
      row_out[tid] = out;
      row_t[tid] = t;
      row_ref[tid] = -INFINITY;
    }
    // scales of the keys of four tiles, requested four tiles ahead
    int raw_k[4] = {}, raw_v[4] = {};
    uint32_t cur_k = 0, cur_v = 0;
    const long long s_row = (static_cast<long long>(b) * p.H_kv + hk) * p.Lk;
    auto request_scales = [&](int i0) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int key = k_begin + (i0 + u) * kKeys + tid;
        raw_k[u] = raw_v[u] = 127;
        if (key < k_end) {
          raw_k[u] = __ldg(p.k_scale + s_row + key);
          raw_v[u] = __ldg(p.v_scale + s_row + key);
        }
      }
    };
    if constexpr (F8) request_scales(0);
    named_barrier(1, 128);
    // Q into shared memory: eight threads per row
    if (n > 0) {
      const int sub = tid & 7;
      for (int r = tid >> 3; r < NR; r += 16) {
        const bool real = r < rows_here;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                          static_cast<long long>(real ? row_out[r] : 0) * p.d);
        if constexpr (F8) {
          constexpr int PER = W / 128;  // 16-element pieces of the row per thread
          uint4 v[PER][2];
          float amax = 0.f;
#pragma unroll
          for (int u = 0; u < PER; ++u) {
            const int c = sub + 8 * u;  // elements 16c .. 16c + 15
            v[u][0] = v[u][1] = make_uint4(0, 0, 0, 0);
            if (real && 16 * c < p.d) {
              v[u][0] = __ldg(src + 2 * c);
              v[u][1] = __ldg(src + 2 * c + 1);
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t q4[4] = {v[u][y].x, v[u][y].y, v[u][y].z, v[u][y].w};
#pragma unroll
              for (int z = 0; z < 4; ++z)
                amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(q4[z])), fabsf(bf16_hi(q4[z]))));
            }
          }
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          // q 2^-e with the largest magnitude in [128, 256)
          const int e = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 7, -100);
          const float inv = pow2i(-e);
          if (sub == 0) row_factor[r] = pow2i(e) * p.scale_log2;
#pragma unroll
          for (int u = 0; u < PER; ++u) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t q4[4] = {v[u][y].x, v[u][y].y, v[u][y].z, v[u][y].w};
              uint32_t a[4], c2[4];
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                const float x0 = bf16_lo(q4[z]) * inv, x1 = bf16_hi(q4[z]) * inv;
                a[z] = pack_e4m3x2(x0, x1);
                const uint32_t h2 = e4m3x2_to_half2(static_cast<uint16_t>(a[z]));
                c2[z] = pack_e4m3x2((x0 - half_lo(h2)) * 32.f, (x1 - half_hi(h2)) * 32.f);
              }
              hi[2 * y] = a[0] | (a[1] << 16);
              hi[2 * y + 1] = a[2] | (a[3] << 16);
              lo[2 * y] = c2[0] | (c2[1] << 16);
              lo[2 * y + 1] = c2[2] | (c2[3] << 16);
            }
            const uint32_t at = sQ + (sub + 8 * u) * (C::NQ * 16) + r * 16;
            st_shared_v4(at, hi[0], hi[1], hi[2], hi[3]);
            st_shared_v4(at + NR * 16, lo[0], lo[1], lo[2], lo[3]);
          }
        } else {
#pragma unroll
          for (int u = 0; u < W / 64; ++u) {
            const int c = sub + 8 * u;  // elements 8c .. 8c + 7
            uint4 v = make_uint4(0, 0, 0, 0);
            if (real && 8 * c < p.d) v = __ldg(src + c);
            st_shared_v4(sQ + c * (C::NQ * 16) + r * 16, v.x, v.y, v.z, v.w);
          }
        }
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(bar(C::Q_FULL));
    named_barrier(1, 128);  // row_factor

    constexpr int GROUPS = NR / 16;
    float l[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) l[r] = 0.f;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const int key = k_begin + i * kKeys + tid;
      float kf = 1.f, ev = 0.f, vinv = 1.f;
      if constexpr (F8) {
        if ((i & 3) == 0) {
          cur_k = raw_k[0] | (raw_k[1] << 8) | (raw_k[2] << 16) | (raw_k[3] << 24);
          cur_v = raw_v[0] | (raw_v[1] << 8) | (raw_v[2] << 16) | (raw_v[3] << 24);
          if (i + 4 < n) request_scales(i + 4);
        }
        const uint32_t kb = (cur_k >> (8 * (i & 3))) & 255u;
        const uint32_t vb = min((cur_v >> (8 * (i & 3))) & 255u, 254u);
        kf = __uint_as_float(kb << 23);
        ev = static_cast<float>(static_cast<int>(vb) - 127);
        vinv = __uint_as_float((254u - vb) << 23);
      }
      // which rows see this key (a tile inside the prefix: all)
      const bool masked = k_begin + (i + 1) * kKeys > min(w.n, k_end);
      uint64_t sees = ~0ull;
      if (masked) {
        if (key >= k_end) {
          sees = 0;
        } else if (key >= w.n) {
          const int j = key - w.n;
          sees = 0;
          for (int r = 0; r < rows_here; ++r) {
            const int t = row_t[r];
            if (t < 0) continue;
            const bool on =
                p.tree_mask
                    ? (__ldg(p.tree_mask + (static_cast<long long>(b) * p.T + t) * p.words + (j >> 6)) >>
                       (j & 63)) & 1
                    : j <= t;
            if (on) sees |= 1ull << r;
          }
        }
      }
      ok = ok && mbar_wait(bar(C::S_FULL + (i & 1)), (i >> 1) & 1, abort_flag, p.status,
                           site + C::S_FULL + (i & 1));
      tc_fence_after();
      // this key's scores
      float s[NR];
      bool over = false;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        if (g * 16 >= rows_here) continue;
        uint32_t c1[16];
        const uint32_t at = t_lane + ((i & 1) ? C::TM_S1 : 0u) + g * 16;
        tmem_ld16(at, c1);
        if constexpr (F8) {
          uint32_t c2[16];
          tmem_ld16(at + NR, c2);
          tmem_ld_wait();
#pragma unroll
          for (int r = 0; r < 16; ++r)
            s[g * 16 + r] = fmaf(fmaf(__uint_as_float(c2[r]), 1.f / 32.f, __uint_as_float(c1[r])),
                                 kf * row_factor[g * 16 + r], ev);
        } else {
          tmem_ld_wait();
#pragma unroll
          for (int r = 0; r < 16; ++r) s[g * 16 + r] = __uint_as_float(c1[r]) * p.scale_log2;
        }
        if (masked) {
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (!((sees >> (g * 16 + r)) & 1)) s[g * 16 + r] = -INFINITY;
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) over |= s[g * 16 + r] > row_ref[g * 16 + r] + C::SLACK;
      }
      tc_fence_before();
      if (any_of_128(over)) {
        // move the references to this tile's maxima and rescale
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          if ((r & ~15) >= rows_here) continue;
          float m = s[r];
#pragma unroll
          for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          if (lane == 0) red[warp * NR + r] = m;
        }
        named_barrier(1, 128);
        // (rows past the block's own, up to the next 16, move along: their
        // scores are 0, not -inf)
        if (tid < NR && (tid & ~15) < rows_here) {
          const float old = row_ref[tid];
          const float m = fmaxf(fmaxf(fmaxf(red[tid], red[NR + tid]), fmaxf(red[2 * NR + tid], red[3 * NR + tid])), old);
          row_alpha[tid] = m == -INFINITY ? 1.f : ex2_approx(old - m);
          row_ref[tid] = m;
        }
        named_barrier(1, 128);
#pragma unroll
        for (int r = 0; r < NR; ++r)
          if ((r & ~15) < rows_here) l[r] *= row_alpha[r];
        if (i > 0) {
          ok = ok && mbar_wait(bar(C::PV_DONE), (i - 1) & 1, abort_flag, p.status, site + C::PV_DONE);
          tc_fence_after();
          for (int c = 0; c < C::BLKS * C::NP; c += 16) {
            if (c % NR >= rows_here) continue;
            uint32_t o[16];
            tmem_ld16(t_lane + C::TM_O + c, o);
            tmem_ld_wait();
#pragma unroll
            for (int r = 0; r < 16; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * row_alpha[c % NR + r]);
            tmem_st16(t_lane + C::TM_O + c, o);
          }
          tmem_st_wait();
          tc_fence_before();
        }
      }
      // P and the V tile's rows past the last key: the previous product must
      // have read P
      if (i > 0) ok = ok && mbar_wait(bar(C::PV_DONE), (i - 1) & 1, abort_flag, p.status, site + C::PV_DONE);
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        if (g * 16 >= rows_here) continue;
        uint32_t w1[8], w2[8], w3[8];
#pragma unroll
        for (int r = 0; r < 16; r += 2) {
          const int a = g * 16 + r;
          const float m0 = row_ref[a], m1 = row_ref[a + 1];
          const float p0 = ex2_approx(s[a] - (m0 == -INFINITY ? 0.f : m0 - C::LIFT));
          const float p1 = ex2_approx(s[a + 1] - (m1 == -INFINITY ? 0.f : m1 - C::LIFT));
          if constexpr (F8) {
            l[a] = fmaf(p0, vinv, l[a]);
            l[a + 1] = fmaf(p1, vinv, l[a + 1]);
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
            l[a] += p0;
            l[a + 1] += p1;
            w1[r >> 1] = pack_bf16x2(p0, p1);
            w2[r >> 1] = pack_bf16x2(p0 - bf16_lo(w1[r >> 1]), p1 - bf16_hi(w1[r >> 1]));
          }
        }
        // 16-byte units [column of units][key]
        if constexpr (F8) {
          const uint32_t at = sP + g * (kKeys * 16) + tid * 16;
          st_shared_v4(at, w1[0], w1[1], w1[2], w1[3]);
          st_shared_v4(at + GROUPS * (kKeys * 16), w2[0], w2[1], w2[2], w2[3]);
          st_shared_v4(at + 2 * GROUPS * (kKeys * 16), w3[0], w3[1], w3[2], w3[3]);
        } else {
          const uint32_t at = sP + 2 * g * (kKeys * 16) + tid * 16;
          st_shared_v4(at, w1[0], w1[1], w1[2], w1[3]);
          st_shared_v4(at + kKeys * 16, w1[4], w1[5], w1[6], w1[7]);
          st_shared_v4(at + 2 * GROUPS * (kKeys * 16), w2[0], w2[1], w2[2], w2[3]);
          st_shared_v4(at + (2 * GROUPS + 1) * (kKeys * 16), w2[4], w2[5], w2[6], w2[7]);
        }
      }
      if (i == n - 1 && k_begin + n * kKeys > k_end) {
        // rows past the last key may hold anything (0 * NaN would be NaN)
        const int it = v_item(i), sl = it % C::SLOTS;
        ok = ok && mbar_wait(bar(C::FULL + sl), (it / C::SLOTS) & 1, abort_flag, p.status, site + C::FULL + sl);
        if (key >= k_end) {
#pragma unroll
          for (int c = 0; c < C::TILE / C::CHUNK; ++c)
#pragma unroll
            for (int u = 0; u < 8; ++u)
              st_shared_v4(s_base + sl * C::TILE + c * C::CHUNK + tid * 128 + u * 16, 0, 0, 0, 0);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(C::P_FULL));
    }

    // ---- epilogue: sums over the keys, then O
    if (n > 0) {
      ok = ok && mbar_wait(bar(C::PV_DONE), (n - 1) & 1, abort_flag, p.status, site + C::PV_DONE);
      tc_fence_after();
    }
    if (*abort_flag) ok = false;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      if ((r & ~15) >= rows_here) continue;
      float t = l[r];
#pragma unroll
      for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      if (lane == 0) red[warp * NR + r] = t;
    }
    named_barrier(1, 128);
    const bool whole = w.active == 1;  // no other split: this is the result
    const long long total_rows = static_cast<long long>(p.B) * p.T * p.H;
    if (tid < rows_here) {
      float L = red[tid] + red[NR + tid] + red[2 * NR + tid] + red[3 * NR + tid];
      float m = row_ref[tid] - C::LIFT;
      if (row_t[tid] < 0 || !ok) {  // an empty row (or a CTA that gave up: an empty partial)
        L = 0.f;
        m = -INFINITY;
      }
      row_alpha[tid] = L > 0.f ? (whole ? 1.f / L : 1.f) : 0.f;
      if (whole) {
        if (p.lse) {
          const int bt = row_out[tid] / p.H, h = row_out[tid] % p.H;
          p.lse[(static_cast<long long>(b) * p.H + h) * p.T + (bt - b * p.T)] =
              L > 0.f ? (m + __log2f(L)) * 0.69314718055994531f : -INFINITY;
        }
      } else {
        p.part_m[split * total_rows + row_out[tid]] = L > 0.f ? m : -INFINITY;
        p.part_l[split * total_rows + row_out[tid]] = L;
      }
    }
    named_barrier(1, 128);
    const int f0 = C::M_O == 64 ? warp * 16 + lane : warp * 32 + lane;
    const bool holds = C::M_O == 128 || lane < 16;
    for (int blk = 0; blk < C::BLKS; ++blk) {
      if (blk * 128 >= p.d) continue;
      const int f = blk * 128 + f0;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        if (g * 16 >= rows_here) continue;
        float o[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) o[r] = 0.f;
        if (n > 0) {
#pragma unroll
          for (int piece = C::PP - 1; piece >= 0; --piece) {
            uint32_t t[16];
            tmem_ld16(t_lane + C::TM_O + blk * C::NP + piece * NR + g * 16, t);
            tmem_ld_wait();
#pragma unroll
            for (int r = 0; r < 16; ++r) o[r] += __uint_as_float(t[r]);
          }
        }
        if (holds && f < p.d) {
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int row = g * 16 + r;
            if (row >= rows_here) break;
            const float a = row_alpha[row];
            const float v = a > 0.f ? o[r] * a : 0.f;
            const long long at = row_out[row];
            if (whole)
              static_cast<__nv_bfloat16*>(p.out)[at * p.d + f] = __float2bfloat16_rn(v);
            else
              p.part_o[(split * total_rows + at) * W + f] = v;
          }
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// One warp per output row: merges the splits' partials of its sequence,
//   o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s,  M = max_s m_s.
template <int W>
__global__ void __launch_bounds__(256) rows_combine_kernel(const __grid_constant__ RowsParams p) {
  constexpr int EPL = W / 32;
  const int lane = static_cast<int>(threadIdx.x & 31);
  const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const long long rows = static_cast<long long>(p.B) * p.T * p.H;
  griddep_wait();  // the split kernel's partials are complete and visible
  if (row >= rows) return;
  const int b = static_cast<int>(row / (static_cast<long long>(p.T) * p.H));
  const int splits = rows_work(p, b).active;
  if (splits == 1) return;  // written by its only split
  float M = -INFINITY;
  for (int s = lane; s < splits; s += 32) M = fmaxf(M, p.part_m[s * rows + row]);
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float L = 0.f;
  float o[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) o[e] = 0.f;
  for (int s = 0; s < splits; ++s) {
    const float ms = p.part_m[s * rows + row];
    if (ms == -INFINITY) continue;  // a split whose keys this row does not see
    const float w = ex2_approx(ms - M);
    L = fmaf(w, p.part_l[s * rows + row], L);
    const float* po = p.part_o + (s * rows + row) * W;
#pragma unroll
    for (int e = 0; e < EPL; ++e)
      if (lane + 32 * e < p.d) o[e] = fmaf(w, po[lane + 32 * e], o[e]);
  }
  const float inv = L > 0.f ? 1.f / L : 0.f;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + row * p.d;
#pragma unroll
  for (int e = 0; e < EPL; ++e)
    if (lane + 32 * e < p.d) dst[lane + 32 * e] = __float2bfloat16_rn(o[e] * inv);
  if (p.lse && lane == 0) {
    const int bt = static_cast<int>(row / p.H), h = static_cast<int>(row % p.H);
    p.lse[(static_cast<long long>(b) * p.H + h) * p.T + (bt - b * p.T)] =
        L > 0.f ? (M + __log2f(L)) * 0.69314718055994531f : -INFINITY;
  }
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
  const int blocks = (p.T * p.G + NR - 1) / NR;
  const dim3 grid(static_cast<unsigned>(p.B * p.H_kv * blocks), static_cast<unsigned>(p.n_splits));
  e = launch_serialized(rows_kernel<F8, W, NR>, grid, dim3(kRowThreads), C::SMEM, stream, p);
  if (e != cudaSuccess) return e;
  int kernels = 1;
  if (p.n_splits > 1) {
    const long long rows = static_cast<long long>(p.B) * p.T * p.H;
    e = launch_serialized(rows_combine_kernel<W>, dim3(static_cast<unsigned>((rows + 7) / 8)), dim3(256),
                          0, stream, p);
    kernels = 2;
  }
  if (info) {
    info->kernels = kernels;
    info->grid = static_cast<int>(grid.x * grid.y);
    info->block = kRowThreads;
    info->smem = C::SMEM;
  }
  return e;
}

// Calls f.template operator()<F8, W, NR>() with the kernel's configuration for
// R rows per key head of d features.
template <typename F>
auto with_config(bool f8, int d, int R, F&& f) {
  if (f8) {
    if (d <= 128) return R <= 16 ? f(RowsCfg<true, 128, 16>{}) : f(RowsCfg<true, 128, 32>{});
    return R <= 16 ? f(RowsCfg<true, 256, 16>{}) : f(RowsCfg<true, 256, 32>{});
  }
  if (d <= 64)
    return R <= 16 ? f(RowsCfg<false, 64, 16>{}) : (R <= 32 ? f(RowsCfg<false, 64, 32>{}) : f(RowsCfg<false, 64, 64>{}));
  if (d <= 128)
    return R <= 16 ? f(RowsCfg<false, 128, 16>{})
                   : (R <= 32 ? f(RowsCfg<false, 128, 32>{}) : f(RowsCfg<false, 128, 64>{}));
  return R <= 16 ? f(RowsCfg<false, 256, 16>{}) : f(RowsCfg<false, 256, 32>{});
}

}  // namespace

int rows_splits(int B, int T, int H, int H_kv, int Lk, int d, bool f8) {
  const int R = T * (H / H_kv);
  return with_config(f8, d, R, [&](auto cfg) {
    using C = decltype(cfg);
    const long long base = static_cast<long long>(B) * H_kv * ((R + C::NR - 1) / C::NR);
    const long long slots = 152ll * C::MIN_BLOCKS;
    const int tiles = (Lk + kKeys - 1) / kKeys;
    // The split count that ends first when every CTA takes its tiles and a
    // start-up worth two: waves of CTAs x (tiles per split + 2).
    int best = 1;
    long long best_cost = -1;
    for (int S = 1; S <= 64 && 2 * (S - 1) <= tiles; ++S) {
      const long long waves = (base * S + slots - 1) / slots;
      const long long cost = waves * ((tiles + S - 1) / S + 2) + (S > 1 ? 2 : 0);
      if (best_cost < 0 || cost < best_cost) {
        best = S;
        best_cost = cost;
      }
    }
    return best;
  });
}

int rows_kernel_width(int d, bool f8) {
  if (f8) return d <= 128 ? 128 : 256;
  return d <= 64 ? 64 : (d <= 128 ? 128 : 256);
}

int rows_box_keys() { return kBoxKeys; }

long long rows_blocks(int B, int T, int H, int H_kv, int d, bool f8) {
  const int R = T * (H / H_kv);
  return with_config(f8, d, R, [&](auto cfg) {
    return static_cast<long long>(B) * H_kv * ((R + decltype(cfg)::NR - 1) / decltype(cfg)::NR);
  });
}

cudaError_t launch_rows(const RowsParams& p, cudaStream_t stream, LaunchInfo* info) {
  return with_config(p.k_scale != nullptr, p.d, p.T * p.G, [&](auto cfg) {
    using C = decltype(cfg);
    return launch_rows_cfg<C::F8, C::W, C::NR>(p, stream, info);
  });
}

}  // namespace mha

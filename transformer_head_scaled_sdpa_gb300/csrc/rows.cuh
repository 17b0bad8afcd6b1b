// What the kernels of a few query rows over a cache share (mha_rows.cu: rows along
// the tensor core's N; mha_rows_block.cu: rows along its M): units of work, waits.
#pragma once

#include "kernels.h"
#include "ptx.cuh"

namespace mha {

constexpr int kKeys = 128;         // keys per tile
constexpr int kBoxKeys = 32;       // keys per small TMA box: a ragged last tile loads only what it needs
constexpr int kSms = 152;
constexpr int kMaxRowSplits = 64;
constexpr int kRoleRowsLoad = 16, kRoleRowsMma = 17, kRoleRowsSoftmax = 18, kRoleRowsQ = 19;

// One arrival for a warp, behind what all its lanes did.
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// The bounded wait of mbar_wait in few instructions: one that runs out raises
// *abort to its site + 1, and the CTA records it in the device status
// at its end.  (Every role waits in many places; with the status's recording in
// each of them the roles' code did not fit the instruction caches, and 40 % of the
// warps' time went to fetching instructions.)
__device__ __forceinline__ bool thread_wait(uint32_t bar, uint32_t parity, volatile int* abort, int site) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) break;
  }
  *abort = site + 1;
  return false;
}
// Whether the phase with this parity has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// By a whole warp with one answer for all lanes.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort, int site) {
  return __all_sync(0xffffffffu, thread_wait(bar, parity, abort, site));
}

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

// ---------------------------------------------------------------------------
// Units
// ---------------------------------------------------------------------------
struct __align__(16) Unit {
  int b;               // sequence (-1: no more units)
  int hk, rb;          // key head, block of rows
  int part;            // number of the (split, sequence): its place in the partials
  int t0, t1;          // its tiles (none: a sequence without keys)
  int n, end;          // keys of the prefix, keys any row may see
  int live;            // drafted tokens of the sequence
  int splits;          // of the sequence (0: no such unit)
  int pad[2];
};
static_assert(sizeof(Unit) == 48, "three 16-byte words");

// A sequence's lengths (clamped): returns the keys that any row may see.
__device__ __forceinline__ int seq_end(const RowsParams& p, int b, int* n, int* live) {
  *n = min(max(__ldg(p.prefix_lens + b), 0), p.Lk);
  *live = p.draft_lens ? min(max(__ldg(p.draft_lens + b), 0), p.T) : p.T;
  return *live == 0 ? 0 : (p.drafts ? min(p.Lk, *n + *live) : *n);
}

// Splits of up to 32 sequences' keys go by one number of tiles for all of them, the
// smallest with which the units fit the launch (p.n_splits per sequence on average):
// a long sequence of a ragged batch then has more splits than a short one, and units
// are of one size.  (5 sequences of 7,001 to 20,000 keys of 256
// features in 8 bits: 36 us, 40 with as many splits for each; 3 of 9,001 to 16,300
// keys, 252 rows: 60 and 63.)  With more sequences the units of
// different sizes even out over the machine, and each is divided by p.n_splits.
constexpr int kBalanced = 32;
__device__ __forceinline__ bool balanced(const RowsParams& p) { return p.n_splits > 1 && p.B <= kBalanced; }

// By a whole warp: lane b has sequence b's first (split, sequence) number and splits;
// *per: tiles of a split.
__device__ __forceinline__ void balance(const RowsParams& p, int lane, int* first, int* splits, int* per) {
  int n, live;
  const int tiles = lane < p.B ? (seq_end(p, lane, &n, &live) + kKeys - 1) / kKeys : 0;
  const int most = __reduce_max_sync(0xffffffffu, tiles), all = __reduce_add_sync(0xffffffffu, tiles);
  const int units = p.n_splits * p.B;
  const int lo = max(1, max((all + units - 1) / units, (most + kMaxRowSplits - 1) / kMaxRowSplits));
  const int hi = max(lo, (most + p.n_splits - 1) / p.n_splits);  // (fits: p.n_splits each)
  const int mine = lane == 31 ? hi : min(hi, lo + lane * ((hi - lo) / 32 + 1));
  int sum = 0;
  for (int b = 0; b < p.B; ++b) sum += max(1, (__shfl_sync(0xffffffffu, tiles, b) + mine - 1) / mine);
  const unsigned fits = __ballot_sync(0xffffffffu, sum <= units);
  *per = __shfl_sync(0xffffffffu, mine, __ffs(fits) - 1);
  *splits = lane < p.B ? max(1, (tiles + *per - 1) / *per) : 0;
  int last = *splits;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, last, o);
    if (lane >= o) last += x;
  }
  *first = last - *splits;
}

// Up to 32 sequences of a launch with more units than can run at once go longest
// first, so that the last units are short ones and the time does not depend on the
// order of the batch.  us, with it and as they come in three orders:
//   8 bits, 16 x 96 heads x 1,024 to 2,048 keys of 128       94.3   93.2 93.2 96.3
//     4 x 96 heads with 16 drafted tokens                    36.5   35.7 36.2 42.0
//     5 x 64 heads x 100 to 2,000 keys, 80 drafted           93.1   99.2 99.7 100
//   bf16, 3 x 96 heads x 500 to 4,000 keys of 128, 5 drafted 55.8   58.6 58.7 60.5
//     4 x 96 heads x 1,024 to 2,048 keys, 25 drafted         56.2   56.0 56.3 57.6
//     rows along M, 3 x 96 heads x 500 to 4,000, 100 drafted 87.6  103.4 110.3 110.3
//     against it: 32 x 40 heads x 30 to 1,000 keys, 8 drafted 63.6  58.7 60.2 61.1
__device__ __forceinline__ bool longest_first(const RowsParams& p, int slots) {
  return p.n_splits == 1 && p.B > 1 && p.B <= kBalanced && static_cast<int>(gridDim.x) > slots;
}

// By a whole warp: the place of sequence `lane` (lanes below B).
__device__ __forceinline__ int place_of(const RowsParams& p, int lane) {
  int n, live, place = 0;
  const int end = lane < p.B ? seq_end(p, lane, &n, &live) : -1;
  for (int b = 0; b < p.B; ++b) {
    const int x = __shfl_sync(0xffffffffu, end, b);
    place += x > end || (x == end && b < lane) ? 1 : 0;
  }
  return place;
}

// Unit `index` of a launch, of sequence b whose keys are in `splits` splits of `per`
// tiles.
__device__ __forceinline__ Unit unit_of(const RowsParams& p, int index, int blocks, int b, int split, int per) {
  Unit w;
  const int u = index % p.units;
  w.hk = blocks == 1 ? u : u / blocks;
  w.rb = u - w.hk * blocks;
  w.part = index / p.units;
  w.b = b;
  w.end = seq_end(p, b, &w.n, &w.live);
  const int tiles = (w.end + kKeys - 1) / kKeys;
  if (per == 0) per = (tiles + p.n_splits - 1) / p.n_splits;  // (not balanced)
  w.splits = per > 0 ? max(1, (tiles + per - 1) / per) : 1;
  if (split >= w.splits) w.splits = 0;
  w.t0 = min(split * per, tiles);
  w.t1 = min(w.t0 + per, tiles);
  return w;
}

// The step of a row or two per key head over a short 8-bit cache (mha_rows_short.cu).
constexpr int kShortRows = 2;    // rows per key head
constexpr int kShortWork = 16384;  // keys x features x rows of a sequence and key head
cudaError_t launch_rows_short(const RowsParams& p, cudaStream_t stream, LaunchInfo* info);

// The rows kernel for many rows per key head of a bf16 cache (mha_rows_block.cu).
constexpr int kBlockRows = 256;  // rows per unit
cudaError_t launch_rows_block(const RowsParams& p, cudaStream_t stream, LaunchInfo* info);

// The step over a 4-bit cache (mha_rows_q4.cu).
struct RowsQ4Shape {
  int width, rows, ctas;  // features a partial row is kept at, rows per unit, CTAs per SM
};
RowsQ4Shape rows_q4_shape(int d, int R);
cudaError_t launch_rows_q4(const RowsParams& p, cudaStream_t stream, LaunchInfo* info);

}  // namespace mha

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

// ---------------------------------------------------------------------------
// Units
// ---------------------------------------------------------------------------
struct __align__(16) Unit {
  int b;               // sequence (-1: no more units)
  int hk, rb, split;   // key head, block of rows, split
  int t0, t1;          // its tiles (none: a sequence without keys)
  int n, end;          // keys of the prefix, keys any row may see
  int live;            // drafted tokens of the sequence
  int splits;          // of the sequence
  int pad[2];
};
static_assert(sizeof(Unit) == 48, "three 16-byte words");

// A sequence's part in a unit: lengths (clamped), tiles per split, splits.
__device__ __forceinline__ void unit_keys(const RowsParams& p, Unit* w) {
  const int n = __ldg(p.prefix_lens + w->b);
  w->n = n < 0 ? 0 : (n > p.Lk ? p.Lk : n);
  w->live = p.T;
  if (p.draft_lens) {
    const int live = __ldg(p.draft_lens + w->b);
    w->live = live < 0 ? 0 : (live > p.T ? p.T : live);
  }
  w->end = w->live == 0 ? 0 : (p.drafts ? min(p.Lk, w->n + w->live) : w->n);
  const int tiles = (w->end + kKeys - 1) / kKeys;
  const int per = (tiles + p.n_splits - 1) / p.n_splits;
  w->splits = per > 0 ? (tiles + per - 1) / per : 1;
  w->t0 = min(w->split * per, tiles);
  w->t1 = min(w->t0 + per, tiles);
}

__device__ __forceinline__ Unit unit_at(const RowsParams& p, int index, int blocks) {
  Unit w;
  const int u = index % p.units, rest = index / p.units;
  w.hk = blocks == 1 ? u : u / blocks;
  w.rb = u - w.hk * blocks;
  w.split = rest / p.B;
  w.b = rest - w.split * p.B;
  unit_keys(p, &w);
  return w;
}

// The rows kernel for many rows per key head of a bf16 cache (mha_rows_block.cu).
constexpr int kBlockRows = 256;  // rows per unit
cudaError_t launch_rows_block(const RowsParams& p, cudaStream_t stream, LaunchInfo* info);

}  // namespace mha

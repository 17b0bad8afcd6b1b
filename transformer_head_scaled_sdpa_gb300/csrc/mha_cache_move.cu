// mha_cache_move.cu -- rows of a key/value cache moved in place, sm_103a: what a
// decoder does with its caches between its steps.
//
//   fork     row (b, j) := row (parent[b], j)        for first[b] <= j < lens[b]
//     (beam search keeps the best continuations, cookipedia article, section
//     "Transformer 全体": a beam that did not survive goes on with another's rows)
//   compact  row (b, prefix[b] + i) := row (b, prefix[b] + path[b, i])  for i < n[b]
//     (of a step's drafted tokens the accepted ones stay, next to the prefix)
//
// All moves read what was there before the call, whatever order they run in and though
// one's source may be another's destination.  A fork keeps positions and a
// compaction keeps sequences, so the byte columns of a cache (one piece of 16 bytes of
// a row, over the sequences or over a sequence's accepted tokens) are independent: a
// block takes a column's moves together, reads all their sources into
// registers, waits for its threads, and writes.  No second buffer, no order, one launch
// for keys, values and scales.
//
// Bound by memory: a fork reads every source row and writes every moved one; a block
// has 32 KB in flight.  A compaction moves a few rows: its time is that of a launch and
// of two dependent reads.
#include "kernels.h"

namespace mha {
namespace {

constexpr int kThreads = 256;
constexpr int kItems = 8;                       // per thread
constexpr int kBlockItems = kThreads * kItems;  // moves of one block at a time

struct Move {
  int to, from;    // sequences (fork), positions after the prefix (compact)
  int first, end;  // fork: positions that move
};

// The largest power of two of columns with which m moves (1 .. kBlockItems) of each are a block's items.
__device__ __forceinline__ int log_columns(int m) { return 31 - __clz(kBlockItems / m); }

// One element of type V for each of `count` items: locate(i, &to, &from) gives its
// addresses, false where nothing moves.  (Asked again for the writes: eight pairs of
// addresses kept beside eight elements took 124 registers.)
template <typename V, typename F>
__device__ __forceinline__ void move_items(int count, F&& locate) {
  V x[kItems];
#pragma unroll
  for (int u = 0; u < kItems; ++u) {
    const int i = static_cast<int>(threadIdx.x) + u * kThreads;
    V* to;
    const V* from;
    // (a coherent load: the source may be written later in this launch)
    if (i < count && locate(i, &to, &from)) x[u] = __ldcg(from);
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kItems; ++u) {
    const int i = static_cast<int>(threadIdx.x) + u * kThreads;
    V* to;
    const V* from;
    if (i < count && locate(i, &to, &from)) *to = x[u];
  }
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------
template <typename S>
__device__ __forceinline__ void fork_scales(const MoveParams& p, const Move* moves, int n, int c, long long e0, int lg,
                                            int lo, int span) {
  S* at = reinterpret_cast<S*>(p.scales[c]);
  const long long all = static_cast<long long>(p.H) * span;
  move_items<S>(n << lg, [&](int i, S** to, const S** from) {
    const Move m = moves[i >> lg];
    const long long e = e0 + (i & ((1 << lg) - 1));
    if (e >= all) return false;
    const long long h = e / span;
    const int j = lo + static_cast<int>(e - h * span);
    if (j < m.first || j >= m.end) return false;
    *to = at + (static_cast<long long>(m.to) * p.H + h) * p.Lk + j;
    *from = at + (static_cast<long long>(m.from) * p.H + h) * p.Lk + j;
    return true;
  });
}

__global__ void __launch_bounds__(kThreads, 4) cache_fork_kernel(const __grid_constant__ MoveParams p) {
  __shared__ Move moves[kMaxForkSeqs];
  __shared__ int count, lowest, highest;
  if (threadIdx.x == 0) {
    count = 0;
    lowest = p.Lk;
    highest = 0;
  }
  __syncthreads();
  griddep_wait();
  for (int b = static_cast<int>(threadIdx.x); b < p.B; b += kThreads) {
    Move m;
    m.to = b;
    m.from = __ldg(p.parent + b);
    m.first = p.first ? max(__ldg(p.first + b), 0) : 0;
    m.end = min(__ldg(p.lens + b), p.Lk);
    if (m.from < 0 || m.from >= p.B || m.from == b || m.first >= m.end) continue;
    moves[atomicAdd(&count, 1)] = m;
    atomicMin(&lowest, m.first);
    atomicMax(&highest, m.end);
  }
  __syncthreads();
  const int n = count;
  if (n == 0) return;
  // a block's columns: 2^lg pieces of the rows of the positions lo .. lo + span - 1, or
  // 2^lg scales of all heads at these positions
  const int lg = log_columns(n), lo = lowest, span = highest - lo;
  const long long pieces = p.row_bytes / 16, all = span * pieces;
  const long long chunks = (all + (1 << lg) - 1) >> lg;
  const long long scale_chunks =
      p.scale_bytes ? (static_cast<long long>(p.H) * span + (1 << lg) - 1) >> lg : 0;
  for (long long x = blockIdx.x; x < 2 * (chunks + scale_chunks); x += gridDim.x) {
    if (x < 2 * chunks) {
      const int c = x >= chunks;
      const long long q0 = lo * pieces + ((c ? x - chunks : x) << lg), stop = (lo + static_cast<long long>(span)) * pieces;
      uint4* at = reinterpret_cast<uint4*>(p.codes[c]);
      const long long seq = p.Lk * pieces;
      move_items<uint4>(n << lg, [&](int i, uint4** to, const uint4** from) {
        const Move m = moves[i >> lg];
        const long long q = q0 + (i & ((1 << lg) - 1));
        if (q >= stop || q < m.first * pieces || q >= m.end * pieces) return false;
        *to = at + m.to * seq + q;
        *from = at + m.from * seq + q;
        return true;
      });
    } else {
      const long long y = x - 2 * chunks;
      const int c = y >= scale_chunks;
      const long long e0 = (c ? y - scale_chunks : y) << lg;
      if (p.scale_bytes == 1) fork_scales<uint8_t>(p, moves, n, c, e0, lg, lo, span);
      else fork_scales<uint32_t>(p, moves, n, c, e0, lg, lo, span);
    }
  }
}

// ---------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------
constexpr int kMaxMoves = 256;      // drafted tokens of a step
constexpr int kMaxPieceLog = 7;     // a block's columns are at most 2 KB of a row

template <typename S>
__device__ __forceinline__ void compact_scales(const MoveParams& p, const Move* moves, int n, int c, long long at0,
                                               int h0, int lg) {
  S* at = reinterpret_cast<S*>(p.scales[c]) + at0;
  move_items<S>(n << lg, [&](int i, S** to, const S** from) {
    const Move m = moves[i >> lg];
    const int h = h0 + (i & ((1 << lg) - 1));
    if (h >= p.H) return false;
    *to = at + static_cast<long long>(h) * p.Lk + m.to;
    *from = at + static_cast<long long>(h) * p.Lk + m.from;
    return true;
  });
}

// Block x of sequence b: its K or V columns x of 2^lg pieces, or the scales of 2^lg heads.
__global__ void __launch_bounds__(kThreads) cache_compact_kernel(const __grid_constant__ MoveParams p, int lg, int chunks,
                                                                 int scale_chunks) {
  __shared__ Move moves[kMaxMoves];
  __shared__ int count;
  if (threadIdx.x == 0) count = 0;
  __syncthreads();
  griddep_wait();
  const int per_seq = 2 * (chunks + scale_chunks);
  const int b = static_cast<int>(blockIdx.x) / per_seq, x = static_cast<int>(blockIdx.x) % per_seq;
  const int prefix = min(max(__ldg(p.first + b), 0), p.Lk);
  const int held = p.lens ? min(max(__ldg(p.lens + b), 0), p.T) : p.T;
  for (int i = static_cast<int>(threadIdx.x); i < held; i += kThreads) {
    const int from = __ldg(p.path + static_cast<long long>(b) * p.T + i);
    // (a token outside the drafted ones, or outside the cache: its row stays as it is)
    if (from < 0 || from >= p.T || from == i || max(from, i) >= p.Lk - prefix) continue;
    Move m;
    m.to = prefix + i;
    m.from = prefix + from;
    m.first = m.end = 0;
    moves[atomicAdd(&count, 1)] = m;
  }
  __syncthreads();
  const int n = count;
  if (n == 0) return;
  if (x < 2 * chunks) {
    const int c = x >= chunks;
    const long long pieces = p.row_bytes / 16, q0 = static_cast<long long>(c ? x - chunks : x) << lg;
    uint4* at = reinterpret_cast<uint4*>(p.codes[c]) + static_cast<long long>(b) * p.Lk * pieces;
    move_items<uint4>(n << lg, [&](int i, uint4** to, const uint4** from) {
      const Move m = moves[i >> lg];
      const long long q = q0 + (i & ((1 << lg) - 1));
      if (q >= pieces) return false;
      *to = at + m.to * pieces + q;
      *from = at + m.from * pieces + q;
      return true;
    });
  } else {
    const int y = x - 2 * chunks, c = y >= scale_chunks, h0 = (c ? y - scale_chunks : y) << lg;
    const long long at0 = static_cast<long long>(b) * p.H * p.Lk;
    if (p.scale_bytes == 1) compact_scales<uint8_t>(p, moves, n, c, at0, h0, lg);
    else compact_scales<uint32_t>(p, moves, n, c, at0, h0, lg);
  }
}

void say(LaunchInfo* info, unsigned grid) {
  if (!info) return;
  info->kernels = 1;
  info->grid = static_cast<int>(grid);
  info->block = kThreads;
  info->smem = 0;
}

// Columns (a power of two) of a compaction's block when up to T tokens move.
int compact_log(int T) {
  int lg = 0;
  while (lg < kMaxPieceLog && (2 << lg) * T <= kBlockItems) ++lg;
  return lg;
}
long long compact_chunks(const MoveParams& p, int lg) { return (p.row_bytes / 16 + (1 << lg) - 1) >> lg; }
long long compact_scale_chunks(const MoveParams& p, int lg) {
  return p.scale_bytes ? (static_cast<long long>(p.H) + (1 << lg) - 1) >> lg : 0;
}

}  // namespace

long long compact_blocks(const MoveParams& p) {
  const int lg = compact_log(p.T);
  return p.B * 2 * (compact_chunks(p, lg) + compact_scale_chunks(p, lg));
}

cudaError_t launch_cache_fork(const MoveParams& p, cudaStream_t stream, LaunchInfo* info) {
  // blocks for every item that the capacity allows, at most eight to an SM: what moves
  // is known on the device alone
  const double items = 2. * p.B * p.Lk * (p.row_bytes / 16 + (p.scale_bytes ? p.H : 0));
  const unsigned most = 152 * 8;
  const unsigned grid = items < static_cast<double>(most) * kBlockItems
                            ? static_cast<unsigned>(items / kBlockItems) + 1
                            : most;
  say(info, grid);
  return launch_serialized(cache_fork_kernel, dim3(grid), dim3(kThreads), 0, stream, p);
}

cudaError_t launch_cache_compact(const MoveParams& p, cudaStream_t stream, LaunchInfo* info) {
  const int lg = compact_log(p.T);
  const unsigned grid = static_cast<unsigned>(compact_blocks(p));
  say(info, grid);
  return launch_serialized(cache_compact_kernel, dim3(grid), dim3(kThreads), 0, stream, p, lg,
                           static_cast<int>(compact_chunks(p, lg)), static_cast<int>(compact_scale_chunks(p, lg)));
}

}  // namespace mha

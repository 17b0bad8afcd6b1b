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
// block takes a column's moves together, has all their sources in shared memory (a fork) or
// registers (a compaction) and its threads at a barrier before it writes one of them.  No
// second buffer, no order, one launch for keys, values and scales.
//
// Bound by memory: a fork reads every source row and writes every moved one, a block with
// two buffers of 32 KB (8-bit, 4 x 4 beams of 96 heads, 280 MB: 53 us, 5.3 TB/s; three
// blocks to an SM; with smaller buffers, which move shorter runs of each row, 16 KB with
// four blocks 69 us, with six 81, when 32 KB took 57; eight elements in each thread's
// registers 81).  A compaction moves a few rows: its time, 2 us, is that of a launch and of
// two dependent reads.
#include "kernels.h"

namespace mha {
namespace {

constexpr int kThreads = 256;
constexpr int kItems = 8;                       // per thread
constexpr int kBlockItems = kThreads * kItems;  // moves of one block at a time
constexpr int kMaxLog = 8;                      // a block's columns: at most a thread each

struct Move {
  int to, from;    // sequences (fork), positions (compact)
  int first, end;  // fork: positions that move
};

// Columns (log2) of a block when m moves (1 .. items) of each are its items.
__host__ __device__ __forceinline__ int log_columns(int m, int items) {
  int lg = 0;
  while (lg < kMaxLog && (2 << lg) * m <= items) ++lg;
  return lg;
}

// All moves of 2^lg columns of elements V.  `column`: the thread's column (threads tid,
// tid + 2^lg, ... share it) of sequence or position 0, `stride` elements between
// sequences or positions; `j`: its position, -1: none moves.
template <typename V>
__device__ __forceinline__ void move_columns(const Move* moves, int n, int lg, V* column, long long stride, int j) {
  V x[kItems];
  const int m0 = static_cast<int>(threadIdx.x) >> lg, step = kThreads >> lg;
#pragma unroll
  for (int u = 0; u < kItems; ++u) {
    if (m0 + u * step >= n) break;
    const Move m = moves[m0 + u * step];
    // (a coherent load: the source may be written later in this launch)
    if (j >= m.first && j < m.end) x[u] = __ldcg(column + m.from * stride);
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kItems; ++u) {
    if (m0 + u * step >= n) break;
    const Move m = moves[m0 + u * step];
    if (j >= m.first && j < m.end) column[m.to * stride] = x[u];
  }
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------
constexpr int kForkBlocks = 3;    // per SM
constexpr int kForkItems = 2048;  // of a block at a time (kMaxForkSeqs at least)
static_assert(kForkItems >= kMaxForkSeqs && kForkItems <= kBlockItems, "a column of every sequence");

template <typename S>
__device__ __forceinline__ void fork_scales(const MoveParams& p, const Move* moves, int n, int lg, int c, long long e,
                                            int lo, int span) {
  // (head e / span, position lo + e % span)
  const long long h = e / span;
  const int j = h < p.H ? lo + static_cast<int>(e - h * span) : -1;
  move_columns(moves, n, lg, reinterpret_cast<S*>(p.scales[c]) + h * p.Lk + max(j, 0),
               static_cast<long long>(p.H) * p.Lk, j);
}

__global__ void __launch_bounds__(kThreads, kForkBlocks) cache_fork_kernel(const __grid_constant__ MoveParams p) {
  extern __shared__ __align__(16) uint8_t held[];  // [2][kForkItems] of 16 bytes, then a move of every sequence
  Move* moves = reinterpret_cast<Move*>(held + 2 * 16 * kForkItems);
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
  // 2^scale_lg scales of all heads at these positions
  const int lg = log_columns(n, kForkItems), scale_lg = log_columns(n, kBlockItems), lo = lowest, span = highest - lo;
  const int own = static_cast<int>(threadIdx.x) & ((1 << lg) - 1);
  const long long pieces = p.row_bytes / 16, seq = p.Lk * pieces;
  const long long chunks = (span * pieces + (1 << lg) - 1) >> lg;
  const long long scale_chunks =
      p.scale_bytes ? (static_cast<long long>(p.H) * span + (1 << scale_lg) - 1) >> scale_lg : 0;
  // The codes by way of shared memory, the next columns' copies while these are written
  // (a thread writes what it copied; the barrier is for the others' rows).
  const uint32_t slots = smem_u32(held) + 16 * threadIdx.x;
  const int m0 = static_cast<int>(threadIdx.x) >> lg, step = kThreads >> lg;
  // The thread's column of chunk x: piece r of position j.  From one chunk to the next they
  // are added to (a division each, twice, was a third of the instructions).
  const long long hop = static_cast<long long>(gridDim.x) << lg;
  const long long hop_j = hop / pieces;
  const long long hop_r = hop - hop_j * pieces;
  long long x = blockIdx.x, j = -1, r = 0;
  int c = -1;
  auto locate = [&]() {  // (x is in keys or values for the first time)
    c = x >= chunks;
    const long long q = ((c ? x - chunks : x) << lg) + own;
    j = q / pieces;
    r = q - j * pieces;
  };
  auto copy = [&](int buffer) {
    uint4* column = nullptr;
    if (x < 2 * chunks) {
      column = reinterpret_cast<uint4*>(p.codes[c]) + (lo + j) * pieces + r;
      const int at = j < span ? lo + static_cast<int>(j) : -1;
      uint32_t to = slots + buffer * (16 * kForkItems);
      for (int i = m0; i < n; i += step, to += 16 * kThreads) {
        const Move m = moves[i];
        if (at >= m.first && at < m.end)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(column + m.from * seq) : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return column;
  };
  locate();
  uint4* column = copy(0);
  int buffer = 0;
  while (x < 2 * chunks) {
    const int at = j < span ? lo + static_cast<int>(j) : -1;
    x += gridDim.x;
    if (c == 0 && x >= chunks) {
      locate();
    } else {
      j += hop_j;
      r += hop_r;
      if (r >= pieces) {
        r -= pieces;
        ++j;
      }
    }
    uint4* next = copy(buffer ^ 1);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    const uint4* from = reinterpret_cast<const uint4*>(held) + buffer * kForkItems + threadIdx.x;
    for (int i = m0; i < n; i += step, from += kThreads) {
      const Move m = moves[i];
      if (at >= m.first && at < m.end) column[m.to * seq] = *from;
    }
    column = next;
    buffer ^= 1;
  }
  for (; x < 2 * (chunks + scale_chunks); x += gridDim.x) {
    const long long y = x - 2 * chunks;
    const int c = y >= scale_chunks;
    const long long e = ((c ? y - scale_chunks : y) << scale_lg) + (threadIdx.x & ((1u << scale_lg) - 1));
    if (p.scale_bytes == 1) fork_scales<uint8_t>(p, moves, n, scale_lg, c, e, lo, span);
    else fork_scales<uint32_t>(p, moves, n, scale_lg, c, e, lo, span);
  }
}

// ---------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------
constexpr int kMaxMoves = 256;  // drafted tokens of a step

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
    m.first = 0;
    m.end = 1;
    moves[atomicAdd(&count, 1)] = m;
  }
  __syncthreads();
  const int n = count;
  if (n == 0) return;
  const int own = static_cast<int>(threadIdx.x) & ((1 << lg) - 1);
  if (x < 2 * chunks) {
    const int c = x >= chunks;
    const long long pieces = p.row_bytes / 16, q = (static_cast<long long>(c ? x - chunks : x) << lg) + own;
    move_columns(moves, n, lg, reinterpret_cast<uint4*>(p.codes[c]) + static_cast<long long>(b) * p.Lk * pieces + q, pieces,
                 q < pieces ? 0 : -1);
  } else {
    const int y = x - 2 * chunks, c = y >= scale_chunks, h = ((c ? y - scale_chunks : y) << lg) + own;
    const long long at = (static_cast<long long>(b) * p.H + h) * p.Lk;
    if (p.scale_bytes == 1) move_columns(moves, n, lg, p.scales[c] + at, 1, h < p.H ? 0 : -1);
    else move_columns(moves, n, lg, reinterpret_cast<uint32_t*>(p.scales[c]) + at, 1, h < p.H ? 0 : -1);
  }
}

void say(LaunchInfo* info, unsigned grid) {
  if (!info) return;
  info->kernels = 1;
  info->grid = static_cast<int>(grid);
  info->block = kThreads;
  info->smem = 0;
}

long long compact_chunks(const MoveParams& p, int lg) { return (p.row_bytes / 16 + (1 << lg) - 1) >> lg; }
long long compact_scale_chunks(const MoveParams& p, int lg) {
  return p.scale_bytes ? (static_cast<long long>(p.H) + (1 << lg) - 1) >> lg : 0;
}

}  // namespace

long long compact_blocks(const MoveParams& p) {
  const int lg = log_columns(p.T, kBlockItems);
  return 2ll * p.B * (compact_chunks(p, lg) + compact_scale_chunks(p, lg));
}

cudaError_t launch_cache_fork(const MoveParams& p, cudaStream_t stream, LaunchInfo* info) {
  // blocks for every item that the capacity allows, at most kForkBlocks to an SM: what moves
  // is known on the device alone
  const double items = 2. * p.B * p.Lk * (p.row_bytes / 16 + (p.scale_bytes ? p.H : 0));
  const unsigned most = 152 * kForkBlocks;
  const unsigned grid = items < static_cast<double>(most) * kBlockItems
                            ? static_cast<unsigned>(items / kBlockItems) + 1
                            : most;
  say(info, grid);
  constexpr int kMostSmem = 2 * 16 * kForkItems + kMaxForkSeqs * static_cast<int>(sizeof(Move));
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static bool attr_set[64] = {};
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(cache_fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  return launch_serialized(cache_fork_kernel, dim3(grid), dim3(kThreads),
                           2 * 16 * kForkItems + p.B * sizeof(Move), stream, p);
}

cudaError_t launch_cache_compact(const MoveParams& p, cudaStream_t stream, LaunchInfo* info) {
  const int lg = log_columns(p.T, kBlockItems);
  const unsigned grid = static_cast<unsigned>(compact_blocks(p));
  say(info, grid);
  return launch_serialized(cache_compact_kernel, dim3(grid), dim3(kThreads), 0, stream, p, lg,
                           static_cast<int>(compact_chunks(p, lg)), static_cast<int>(compact_scale_chunks(p, lg)));
}

}  // namespace mha

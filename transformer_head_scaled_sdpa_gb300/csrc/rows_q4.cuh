// rows_q4.cuh -- what the kernels of the steps over the 4-bit cache share
// (mha_rows_q4.cu: up to sixteen rows per key head; mha_rows_q4_many.cu: more).
#pragma once

#include "fp8.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace mha {

// Codes are fp16 subnormals to the tensor cores, c 2^-24, exact; but their products are aligned
// by the factors' exponents, a subnormal's as 2^-14, and of the sixteen that are added at a time
// each is cut 25 places below the largest: at 2^-15 of the largest q (or weight) of the sixteen,
// times a code of 1.  (Measured, on mma.sync and tcgen05 alike.)  A q within 2^8 of that largest
// loses nothing, having eight bits; an output loses less than 16 x 2^-15 of the largest weight
// times its step for each sixteen keys, as much as fp16 takes from the weight.  Codes made normal numbers by a product
// more per two of them lose nothing there, and time: 16 x 96 heads x 1,024 to 2,048 keys 59.9 to
// 64.0 us, 4 x 96 heads x 16 rows 35.1 to 38.0, 8 x 24 heads x 56 rows 68.1 to 70.5.
constexpr float kNoRef = -3.0e38f;  // a row that has seen no key
constexpr float kLift = 8.f;        // weights are 2^kLift at their reference
constexpr float kLimit = 15.f;      // and stay below 2^kLimit, inside fp16's range
// (A reference is a score less kLift.  Scores near 2^27 have places of 16, and to the nearest of
// them a reference could lie 16 below its score: it is rounded up.)
__device__ __forceinline__ float lifted(float m) { return __fadd_ru(m, -kLift); }

// Swizzle of TMA's rows of W / 2 bytes (32, 64 or 128): 16-byte piece c of row `key` of a
// tile lies at piece c ^ swizzle(key), so that the eight rows of a matrix lie in
// different banks.
template <int W>
__device__ __forceinline__ int swizzle(int key) {
  return W == 64 ? (key >> 2) & 1 : (W == 128 ? (key >> 1) & 3 : key & 7);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Queries are scaled by powers of two, 2^-e to a row.  A row's factor, 2^(e + 24) times the
// scale, would pass float32's range from |q| = 2^118 / scale on, though its scores be finite:
// for a unit with a factor above 2^100 (top: the largest e of its finite rows) all factors are
// taken 2^shift smaller and the keys' steps and offsets as much larger.  These stay in
// range: the scores of that largest row are finite (include/mha.h has the bound).
__device__ __forceinline__ int factor_shift(int top, float scale_log2) {
  const int exponent = static_cast<int>(__float_as_uint(scale_log2) >> 23) - 127;
  return min(max(top + 24 + exponent - 100, 0), 100);
}

// What a key's offset and step, and its value's, come to in a step.  A value's pair that is
// not finite (the write's NaN offset; a step of 0 is as much) makes the scores NaN, and its
// factors are 0: a row that sees the position is then NaN in out and in lse, and one that does
// not has no score of it and the weight 0, which meets nothing but finite factors and codes.
struct KeyFactors {
  float step, lo;             // of the key
  float v_log, v_inv, v_ofs;  // of the value: log2 step, 1 / step, lo / step
};
// (key_scale: 2^shift)
__device__ __forceinline__ KeyFactors key_factors(uint32_t k, uint32_t v, float key_scale) {
  KeyFactors f;
  f.step = bf16_hi(k) * key_scale;
  f.lo = bf16_lo(k) * key_scale;
  const float step = bf16_hi(v);
  f.v_log = lg2_approx(step);
  f.v_inv = rcp_approx(step);
  f.v_ofs = bf16_lo(v) * f.v_inv;
  if (!(fabsf(f.v_ofs) < INFINITY)) {
    f.v_log = __int_as_float(0x7fc00000);
    f.v_inv = f.v_ofs = 0.f;
  }
  return f;
}

// This CTA's unit of a launch whose sequences' units are of `blocks` blocks of rows;
// false when it has none.
__device__ __forceinline__ bool this_unit(const RowsParams& p, int blocks, int slots, int lane, Unit* unit) {
  const int index = static_cast<int>(blockIdx.x), part = index / p.units;
  if (balanced(p)) {
    int first, splits, per;
    balance(p, lane, &first, &splits, &per);
    const unsigned here = __ballot_sync(0xffffffffu, lane < p.B && part >= first && part < first + splits);
    if (here == 0) return false;  // (more units than the sequences have splits)
    const int b = __ffs(here) - 1;
    *unit = unit_of(p, index, blocks, b, part - __shfl_sync(0xffffffffu, first, b), __shfl_sync(0xffffffffu, per, 0));
  } else if (longest_first(p, slots)) {
    const int place = place_of(p, lane);
    const unsigned here = __ballot_sync(0xffffffffu, lane < p.B && place == part);
    *unit = unit_of(p, index, blocks, __ffs(here) - 1, 0, 0);
  } else {
    *unit = unit_of(p, index, blocks, part % p.B, part / p.B, 0);
  }
  return unit->splits > 0;
}

// Word x % 4 of the mask of row x / 4 (a chain's: bits 0 .. t).
template <typename F>
__device__ __forceinline__ uint64_t mask_word(const RowsParams& p, const Unit& it, int x, F&& out_row) {
  int t;
  const int out = out_row(x >> 2, &t), word = x & 3;
  if (out < 0 || t >= it.live || it.end <= it.n) return 0;
  if (p.tree_mask)
    return word < p.words ? __ldg(p.tree_mask + (static_cast<long long>(it.b) * p.T + t) * p.words + word) : 0;
  const int count = t + 1 - 64 * word;
  return count >= 64 ? ~0ull : (count <= 0 ? 0ull : (1ull << count) - 1);
}

// Whether a row sees a key, for a thread that has a key and many rows: a row's mask (uint64 [4]
// in shared memory) is read as words of 32 bits, the key's word and bit found once for all rows,
// and nothing branches per row (64 sequences of 70 to 190 keys, 63 drafted tokens of 32 / 8
// heads of 128: 165 us, 177 with the mask's 64 bits shifted row by row, 222 with branches).
struct KeyMask {
  uint32_t bit, all;  // of the word (0: no row sees the key); ~0: every row does, the key is the prefix's
  int word;
  __device__ __forceinline__ KeyMask(int key, int stop, int prefix) {
    const int off = key - prefix;  // (of a key that rows may see below 256: drafted tokens end there)
    all = off < 0 ? 0xffffffffu : 0u;
    bit = key < stop ? 1u << (off & 31) : 0u;
    word = (off >> 5) & 7;
  }
  __device__ __forceinline__ bool seen_by(const uint64_t (*masks)[4], int row) const {
    return ((reinterpret_cast<const uint32_t*>(masks[row])[word] | all) & bit) != 0;
  }
};

// The offsets and steps of the key and the value that a thread owns in each tile, copied
// into shared memory kAhead tiles ahead.  (Loaded into registers, even a tile ahead, they
// were waited for within the tile: the hardware counts a warp's outstanding operations in
// a few counters, and one that other, short operations shared with them was not empty
// before they had come: 1,500 of a tile's 2,600 cycles.)
constexpr int kAhead = 3;
struct Scales {
  static constexpr int BYTES = (kAhead + 1) * 128 * 8;
  uint32_t at;               // the thread's slot 0
  const uint32_t *k, *v;     // of position 0
  int own, stop;             // the thread's key of a tile; keys past `stop` are its last one
  __device__ __forceinline__ void copy(int i, int tile0) const {
    if (tile0 < stop) {
      const int key = min(tile0 + own, stop - 1);
      const uint32_t to = at + (i & kAhead) * 1024;
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(k + key) : "memory");
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + 4), "l"(v + key) : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __device__ __forceinline__ void start(int first) const {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) copy(i, first + i * kKeys);
  }
  // Tile i's words (its place in the unit), and the copy of tile i + kAhead's.
  __device__ __forceinline__ uint2 get(int i, int tile0) const {
    copy(i + kAhead, tile0 + kAhead * kKeys);
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
    uint2 w;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w.x), "=r"(w.y) : "r"(at + (i & kAhead) * 1024) : "memory");
    return w;
  }
};
static_assert((kAhead & (kAhead + 1)) == 0, "slots by a mask");

// What a CTA loads: tiles of kKeys keys or values.
template <int W>
struct Loader {
  static constexpr int ROW = W / 2, TILE = kKeys * ROW;
  const RowsParams& p;
  const Unit& it;
  int stop;
  // (a ragged tile in boxes of kRowsQ4Box keys as far as it goes; what lies behind in the
  // ring are some codes: finite, and their weights are 0)
  __device__ __forceinline__ int boxes(int key) const {
    return stop - key >= kKeys ? 0 : (stop - key + kRowsQ4Box - 1) / kRowsQ4Box;
  }
  __device__ __forceinline__ uint32_t bytes(int key) const {
    const int n = boxes(key);
    return n == 0 ? TILE : n * kRowsQ4Box * ROW;
  }
  __device__ __forceinline__ void copy(uint32_t dst, uint32_t bar, int key, bool v) const {
    const int n = boxes(key);
    if (n == 0) {
      tma_load_4d(dst, v ? &p.tm_v : &p.tm_k, bar, 0, it.hk, key, it.b);
      return;
    }
#pragma unroll 1
    for (int x = 0; x < n; ++x)
      tma_load_4d(dst + x * kRowsQ4Box * ROW, v ? &p.tm_v_box : &p.tm_k_box, bar, 0, it.hk, key + x * kRowsQ4Box, it.b);
  }
  // Keys and values side by side.
  __device__ __forceinline__ void operator()(uint32_t dst, uint32_t bar, int key) const {
    mbar_arrive_expect_tx(bar, 2 * bytes(key));
    copy(dst, bar, key, false);
    copy(dst + TILE, bar, key, true);
  }
};

// The packed tiles of a unit in the order in which mha_rows_q4_many.cu loads them: K0 K1 V0 K2
// V1 ..., item x to slot x % slots of its ring.
struct RingItems {
  int slots, tiles;
  __host__ __device__ int slot(int x) const { return x % slots; }
  __host__ __device__ int keys(int t) const { return t == 0 ? 0 : 2 * t - 1; }
  __host__ __device__ int values(int t) const { return t + 1 < tiles ? 2 * t + 2 : 2 * t + 1; }
  __host__ __device__ bool is_values(int x) const { return x == 2 * tiles - 1 || (x > 0 && (x & 1) == 0); }
  __host__ __device__ int tile(int x) const {
    return x == 2 * tiles - 1 ? tiles - 1 : (is_values(x) ? x / 2 - 1 : (x + 1) / 2);
  }
};
// Keys and values are emptied by warps of their own, and a slot has a barrier for each of the
// two: a wait by parity cannot tell a phase from the one before the last, so who waits on a
// barrier must have waited for each of its phases.  The parities of one of the two, a bit to
// a slot, turned with every item:
struct SlotParity {
  uint32_t bits = 0;
  __host__ __device__ int next(int slot) {
    const int parity = static_cast<int>(bits >> slot) & 1;
    bits ^= 1u << slot;
    return parity;
  }
  __host__ __device__ int last(int slot) const { return static_cast<int>(~bits >> slot) & 1; }
};

// More than sixteen rows per key head (mha_rows_q4_many.cu).
RowsQ4Shape rows_q4_many_shape(int d, int R);
cudaError_t launch_rows_q4_many(const RowsParams& p, cudaStream_t stream, LaunchInfo* info);

}  // namespace mha

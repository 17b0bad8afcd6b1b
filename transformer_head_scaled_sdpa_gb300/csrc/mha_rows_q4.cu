// mha_rows_q4.cu -- attention of a few query rows per sequence over the 4-bit
// key/value cache (the decode step and the step of a tree of drafted tokens),
// sm_103a.
//
// A cached row of a key head is x = lo + step * c with codes c = 0 .. 15 (q4.cuh), so
//   s_jr = scale q_r . k_j = scale (stepk_j (q_r . c_j) + lok_j sum_f q_rf)
//   o_r  = sum_j a_jr v_j  = sum_j (a_jr stepv_j) (c_j + lov_j / stepv_j)
// and both products are of the codes alone, with a key's offset and step applied to
// its scores and weights.  The softmax keeps w_jr = 2^(s_jr + log2 stepv_j - m_r): the
// products take w, the denominator adds w / stepv, the offsets' share of the output is
// the row's sum of w lov / stepv.
//
// The codes go from global memory to registers and from there to the tensor core as
// they lie: four bits in the low bits of an fp16 are the subnormal c 2^-24, exact, so
// unpacking is a mask (one per two codes, and a shift per eight; the odd nibbles stay 16
// times too large, and q, or the output, is divided by 16 there).  Each lane loads the
// part of a row that its fragment wants:
//   S^T [16 keys x 8 rows] = K [16 x d] Q^T: lane (g, j) of a warp has the j-th quarter
//     of the rows of keys g and g + 8; the order of the features along the reduction
//     is free, and Q is laid out in the same one.
//   O^T [16 features x 8 rows] += V^T [16 x 16 keys] P^T: lane (g, j) has the g-th
//     eighth of the rows of keys 2j, 2j + 1, 2j + 8, 2j + 9; two keys' bytes are brought
//     together by one byte permutation, and their low and high nibbles are the
//     fragment's two features.
// The weights' fragment is the scores' transposed (movmatrix).  Nothing passes through
// shared memory but the four warps' merge at the end of a unit, and no warp waits for
// another before that.
//
// mma.sync and not tcgen05: reading the cache bounds a step of a few rows (68 bytes per
// row of 128 features), and tcgen05's operands lie in shared memory in 8 bits or more:
// copying the packed tile there, reading it, writing the unpacked tile and reading that
// are 6 bytes of shared-memory traffic per cached byte, at the rate of HBM more than
// the 128 bytes a clock that an SM has.
//
// q is scaled by a power of two to [2^14, 2^15) at its row's largest and then exact in
// fp16 (to 2^-40 of that); the weights are rounded to fp16 (2^-11 relative); products,
// the denominator and the offsets' sums are float32.  The reference m of a row moves when a
// tile's largest weight passes it by more than 2^kSlack.
#include <cuda_bf16.h>

#include "fp8.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace mha {
namespace {

constexpr int kWarps = 4;
constexpr int kTile = kRowsQ4Keys;  // keys of a warp's tile
constexpr float kLift = 8.f;        // weights are 2^kLift at their reference
constexpr float kSlack = 7.f;       // and stay below 2^(kLift + kSlack), inside fp16's range
constexpr float kNoRef = -3.0e38f;  // a row that has seen no key
constexpr int kRoleRowsQ4 = 20;

// W: widest head; NT: blocks of 8 rows; FEW: a row or two, whose columns hold four
// parts of the keys each; ST: tiles in a warp's ring; CTAS: per SM.
template <int W_, int NT_, bool FEW_, int ST_, int CTAS_>
struct Q4Cfg {
  static constexpr int W = W_, NT = NT_, ST = ST_, CTAS = CTAS_;
  static constexpr bool FEW = FEW_;
  static_assert(!FEW || NT == 1, "one block of columns");
  static constexpr int NR = FEW ? 2 : 8 * NT;  // rows of a unit
  static constexpr int ROW = W / 2;            // bytes of a tile's row
  static constexpr int KW = W / 32;            // words of a key's row per lane
  static constexpr int VW = W / 64;            // words of a value's row per lane
  static constexpr int FT = W / 16;            // blocks of 16 features
  static constexpr bool Q_SHARED = W * NT > 128;  // Q's fragments in shared memory
  // merge: a warp's row of sums, eight lanes' features 4 floats apart
  static constexpr int GS = W / 8 + 4, RS = 8 * GS + 2;
  static constexpr int TILE = kTile * ROW;     // bytes of a tile's keys, and of its values
  static constexpr int RING = ST * 2 * TILE;   // a warp's; its sums at the end
  static_assert(RING >= 8 * RS * 4 && RING % 1024 == 0, "ring");
  static constexpr int OFF_BAR = kWarps * RING;                  // [warp][stage]
  static constexpr int OFF_ABORT = OFF_BAR + kWarps * ST * 8;
  static constexpr int OFF_MASKS = (OFF_ABORT + 4 + 15) / 16 * 16;  // uint64 [NR][4]
  static constexpr int OFF_STATS = OFF_MASKS + NR * 32;          // float [warp][NR][3]
  static constexpr int OFF_KEYS = (OFF_STATS + kWarps * NR * 12 + 15) / 16 * 16;  // float4 [warp][32], float [warp][32]
  static constexpr int OFF_Q = OFF_KEYS + (FEW ? 0 : kWarps * kTile * 20);        // uint2 [2 KW NT][32]
  static constexpr int SMEM = OFF_Q + (Q_SHARED ? 2 * KW * NT * 256 : 0) + 1024;
};

// Where row g of a block of 8 scores lies in its block of 8 keys.  A lane of scores
// (g, j) reads the key of row g, one of values the keys of rows 2 j and 2 j + 1; in
// this order neither reads two rows out of the same banks at once (W 64: rows of 32
// bytes as they are; 128: of 64, TMA's 64-byte swizzle; 256: of 128, the 128-byte one).
template <int W>
__device__ __forceinline__ int key_of_row(int g) {
  constexpr uint32_t order = W == 64 ? 0x53427160u : (W == 128 ? 0x65217430u : 0x36147250u);
  return static_cast<int>((order >> (4 * g)) & 7u);
}
// Byte `at` of row `key` of a tile as TMA wrote it.
template <int W>
__device__ __forceinline__ uint32_t tile_at(int key, int at) {
  const int chunk = W == 64 ? at >> 4 : (W == 128 ? (at >> 4) ^ ((key >> 1) & 3) : (at >> 4) ^ (key & 7));
  return static_cast<uint32_t>(key * (W / 2) + chunk * 16 + (at & 15));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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

// N consecutive words of shared memory.
template <int N>
__device__ __forceinline__ void ld_shared(uint32_t at, uint32_t* w) {
  if constexpr (N == 1) {
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at) : "memory");
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
  } else {
    static_assert(N == 4, "words");
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(at)
                 : "memory");
  }
}

// What a key's offset and step, and its value's, come to in a step.
struct KeyFactors {
  float step, lo;         // of the key
  float v_log, v_inv, v_ofs;  // of the value: log2 step, 1 / step, lo / step
};
__device__ __forceinline__ KeyFactors key_factors(uint32_t k, uint32_t v) {
  KeyFactors f;
  f.step = bf16_hi(k);
  f.lo = bf16_lo(k);
  const float step = bf16_hi(v);
  f.v_log = lg2_approx(step);
  f.v_inv = __frcp_rn(step);
  f.v_ofs = bf16_lo(v) * f.v_inv;
  return f;
}

template <class C>
__global__ void __launch_bounds__(32 * kWarps, C::CTAS) rows_q4_kernel(const __grid_constant__ RowsParams p) {
  constexpr int W = C::W, NT = C::NT, KW = C::KW, VW = C::VW, FT = C::FT, NR = C::NR;
  constexpr bool FEW = C::FEW;
  constexpr int MT = kTile / 16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
  uint64_t(*masks)[4] = reinterpret_cast<uint64_t(*)[4]>(smem + C::OFF_MASKS);
  float(*stats)[NR][3] = reinterpret_cast<float(*)[NR][3]>(smem + C::OFF_STATS);
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int g = lane >> 2, j = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * C::RING;
  const uint32_t bars = smem_u32(smem) + C::OFF_BAR + warp * C::ST * 8;
  if (lane == 0) {
    for (int s = 0; s < C::ST; ++s) mbar_init(bars + 8 * s, 1);
    if (warp == 0) *abort_flag = 0;
    fence_mbar_init();
  }
  __syncwarp();
  griddep_wait();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- this CTA's unit
  const int n_rows = p.T * p.G;
  const int blocks = (n_rows + NR - 1) / NR;
  const int index = static_cast<int>(blockIdx.x), part = index / p.units;
  Unit it;
  if (balanced(p)) {
    int first, splits, per;
    balance(p, lane, &first, &splits, &per);
    const unsigned here = __ballot_sync(0xffffffffu, lane < p.B && part >= first && part < first + splits);
    if (here == 0) return;  // (more units than the sequences have splits)
    const int b = __ffs(here) - 1;
    it = unit_of(p, index, blocks, b, part - __shfl_sync(0xffffffffu, first, b), __shfl_sync(0xffffffffu, per, 0));
  } else if (longest_first(p, kSms * C::CTAS)) {
    const int place = place_of(p, lane);
    const unsigned here = __ballot_sync(0xffffffffu, lane < p.B && place == part);
    it = unit_of(p, index, blocks, __ffs(here) - 1, 0, 0);
  } else {
    it = unit_of(p, index, blocks, part % p.B, part / p.B, 0);
  }
  if (it.splits == 0) return;

  // ---- a warp's tiles: keys first + 32 warp .., every 128; two copies of each in flight
  const int stop = min(it.t1 * kKeys, it.end);
  const int first = it.t0 * kKeys + warp * kTile;
  auto request = [&](int key, int stage) {
    const uint32_t bar = bars + 8 * stage, dst = ring + stage * 2 * C::TILE;
    const int rows = min(kTile, stop - key);
    if (rows == kTile) {
      mbar_arrive_expect_tx(bar, 2 * C::TILE);
      tma_load_4d(dst, &p.tm_k, bar, 0, it.hk, key, it.b);
      tma_load_4d(dst + C::TILE, &p.tm_v, bar, 0, it.hk, key, it.b);
    } else {
      // a ragged one in boxes of kRowsQ4Box keys as far as it goes (what lies behind in
      // the ring are some codes: finite, and their weights are 0)
      const int boxes = (rows + kRowsQ4Box - 1) / kRowsQ4Box;
      mbar_arrive_expect_tx(bar, 2 * boxes * kRowsQ4Box * C::ROW);
      for (int x = 0; x < boxes; ++x) {
        const uint32_t to = dst + x * kRowsQ4Box * C::ROW;
        tma_load_4d(to, &p.tm_k_box, bar, 0, it.hk, key + x * kRowsQ4Box, it.b);
        tma_load_4d(to + C::TILE, &p.tm_v_box, bar, 0, it.hk, key + x * kRowsQ4Box, it.b);
      }
    }
  };
  if (lane == 0)
    for (int s = 0; s < C::ST; ++s)
      if (first + s * kKeys < stop) request(first + s * kKeys, s);
  // lane's key's offsets and steps, a tile ahead (keys past the end: the last one's)
  const long long scales = (static_cast<long long>(it.b) * p.H_kv + it.hk) * p.Lk;
  const uint32_t* k_scale = reinterpret_cast<const uint32_t*>(p.k_scale) + scales;
  const uint32_t* v_scale = reinterpret_cast<const uint32_t*>(p.v_scale) + scales;
  // (lane (g, j) has row g of block j of 8 keys)
  const int own = 8 * j + key_of_row<W>(g);
  uint32_t ks = 0, vs = 0;
  if (first < stop) {
    const int key = min(first + own, stop - 1);
    ks = __ldg(k_scale + key);
    vs = __ldg(v_scale + key);
  }

  // Output row of row r of the unit (-1 past the last), t: its drafted token.
  auto out_row = [&](int r, int* t) {
    const int gr = it.rb * NR + r;
    *t = -1;
    if (gr >= n_rows) return -1;
    *t = p.G == 1 ? gr : gr / p.G;
    return (it.b * p.T + *t) * p.H + it.hk * p.G + (gr - *t * p.G);
  };

  // ---- Q: lane (g, j) holds the features of its part of the keys' rows, of the row of
  // column 8 n + g (FEW: the even columns are row 0, the odd ones row 1)
  uint2 q[C::Q_SHARED ? 1 : 2 * KW * NT];
  uint2* q_shared = reinterpret_cast<uint2*>(smem + C::OFF_Q) + lane;
  float fa[NT][2], fb[NT][2];  // factors of a row's product and of its sum: columns 8 n + 2 j, + 1
  constexpr int KV = KW > 4 ? 4 : KW;  // words loaded at once: 16 j .. (256 wide: and 64 + 16 j ..)
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    int t;
    const int out = out_row(FEW ? g & 1 : 8 * n + g, &t);
    const bool live = out >= 0 && t < it.live;
    const uint16_t* src = static_cast<const uint16_t*>(p.q) + static_cast<long long>(max(out, 0)) * p.d;
    uint4 v[KW];
    float amax = 0.f;
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      const int f = (w / KV) * 128 + 8 * KV * j + 8 * (w % KV);
      v[w] = make_uint4(0, 0, 0, 0);
      if (live && f < p.d) v[w] = __ldg(reinterpret_cast<const uint4*>(src + f));
      const uint32_t x[4] = {v[w].x, v[w].y, v[w].z, v[w].w};
#pragma unroll
      for (int y = 0; y < 4; ++y) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(x[y])), fabsf(bf16_hi(x[y]))));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // q 2^-e with the largest magnitude in [2^14, 2^15)
    const int e = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 14, -100);
    const float inv = pow2i(-e);
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      const float y[8] = {bf16_lo(v[w].x) * inv, bf16_hi(v[w].x) * inv, bf16_lo(v[w].y) * inv, bf16_hi(v[w].y) * inv,
                          bf16_lo(v[w].z) * inv, bf16_hi(v[w].z) * inv, bf16_lo(v[w].w) * inv, bf16_hi(v[w].w) * inv};
#pragma unroll
      for (int x = 0; x < 8; ++x) sum += y[x];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint2 b = make_uint2(pack_f16x2(y[2 * h], y[4 + 2 * h]),
                                   pack_f16x2(y[2 * h + 1] * 0.0625f, y[5 + 2 * h] * 0.0625f));
        if constexpr (C::Q_SHARED) {
          if (warp == 0) q_shared[((2 * w + h) * NT + n) * 32] = b;
        } else {
          q[(2 * w + h) * NT + n] = b;
        }
      }
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    const float f = pow2i(e) * p.scale_log2;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int from = FEW ? 4 * r : 8 * j + 4 * r;
      fa[n][r] = __shfl_sync(0xffffffffu, f * 16777216.f, from);
      fb[n][r] = __shfl_sync(0xffffffffu, f * sum, from);
    }
  }
  // the rows' mask words (a chain's: bits 0 .. t)
  for (int x = static_cast<int>(threadIdx.x); x < NR * 4; x += 32 * kWarps) {
    int t;
    const int out = out_row(x >> 2, &t), word = x & 3;
    uint64_t bits = 0;
    if (out >= 0 && t < it.live && it.end > it.n) {
      if (p.tree_mask) {
        if (word < p.words) bits = __ldg(p.tree_mask + (static_cast<long long>(it.b) * p.T + t) * p.words + word);
      } else {
        const int count = t + 1 - 64 * word;
        bits = count >= 64 ? ~0ull : (count <= 0 ? 0ull : (1ull << count) - 1);
      }
    }
    masks[x >> 2][word] = bits;
  }
  __syncthreads();

  float o[NT][FT][4];
  float ref[NT][2], l[NT][2], ofs[NT][2];  // references less kLift
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int f = 0; f < FT; ++f)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[n][f][x] = 0.f;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      ref[n][r] = kNoRef;
      l[n][r] = 0.f;
      ofs[n][r] = 0.f;
    }
  }
  // lane's places in a tile: the key of row g, the values of rows 2 j and 2 j + 1
  uint32_t k_at[KW / KV], v_at[2];
#pragma unroll
  for (int w = 0; w < KW / KV; ++w) k_at[w] = tile_at<W>(key_of_row<W>(g), 64 * w + 4 * KV * j);
#pragma unroll
  for (int x = 0; x < 2; ++x) v_at[x] = C::TILE + tile_at<W>(key_of_row<W>(2 * j + x), 4 * VW * g);
  float4* keys = reinterpret_cast<float4*>(smem + C::OFF_KEYS) + warp * kTile;
  float* keys_ofs = reinterpret_cast<float*>(smem + C::OFF_KEYS + kWarps * kTile * 16) + warp * kTile;

  bool ok = true;
  int stage = 0;
  uint32_t parity = 0;
#pragma unroll 1
  for (int key0 = first; key0 < stop; key0 += kKeys) {
    const uint32_t tile = ring + stage * 2 * C::TILE;
    ok = __all_sync(0xffffffffu, mbar_wait(bars + 8 * stage, parity, abort_flag, p.status, kRoleRowsQ4 * 64 + stage));
    if (!ok) break;
    // ---- scores: s[n][m] = keys of rows g, 8 + g of block m, columns 2 j, 2 j + 1 of block n
    float s[NT][MT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[n][m][x] = 0.f;
#pragma unroll
    for (int w0 = 0; w0 < KW; w0 += KV) {
      uint32_t kc[MT][2][KV];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) ld_shared<KV>(tile + k_at[w0 / KV] + (16 * m + 8 * h) * C::ROW, kc[m][h]);
#pragma unroll
      for (int w = 0; w < KV; ++w)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint2 b[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const int i = (2 * (w0 + w) + h) * NT + n;
            if constexpr (C::Q_SHARED) b[n] = q_shared[i * 32];
            else b[n] = q[i];
          }
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const uint32_t x0 = h ? kc[m][0][w] >> 8 : kc[m][0][w], x1 = h ? kc[m][1][w] >> 8 : kc[m][1][w];
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma_f16(s[n][m], x0 & 0x000f000fu, x1 & 0x000f000fu, x0 & 0x00f000f0u, x1 & 0x00f000f0u, b[n].x, b[n].y);
          }
        }
    }
    // ---- weights
    const KeyFactors mine = key_factors(ks, vs);
    if (key0 + kKeys < stop) {
      const int key = min(key0 + kKeys + own, stop - 1);
      ks = __ldg(k_scale + key);
      vs = __ldg(v_scale + key);
    }
    const bool masked = key0 + kTile > min(it.n, stop);
    uint32_t pt[NT][MT][2];  // weights transposed: column g, keys of rows 2 j, 2 j + 1 (+ 8)
    if constexpr (FEW) {
      // every column pair has all the keys' scores: lane (g, j) takes those of its own key
      float x[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float lo = j & 1 ? s[0][0][2 + r] : s[0][0][r], hi = j & 1 ? s[0][1][2 + r] : s[0][1][r];
        x[r] = fmaf((j & 2 ? hi : lo) * fa[0][r], mine.step, fmaf(fb[0][r], mine.lo, mine.v_log));
      }
      float v_inv = mine.v_inv, v_ofs = mine.v_ofs;
      if (masked) {
        const int key = key0 + own, off = key - it.n;
        bool any = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          bool sees = key < stop;
          if (sees && off >= 0) sees = (masks[r][off >> 6] >> (off & 63)) & 1;  // (off < 256: drafted tokens end there)
          if (!sees) x[r] = -INFINITY;
          any = any || sees;
        }
        // (what hides from both may hold anything, and 0 * NaN would be NaN)
        if (!any) v_inv = v_ofs = 0.f;
      }
      if (__any_sync(0xffffffffu, fmaxf(x[0] - ref[0][0], x[1] - ref[0][1]) > kLift + kSlack)) {
        // references up to this tile's maxima, what was summed down by as much
        float by[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float m = x[r];
#pragma unroll
          for (int z = 1; z < 32; z <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, z));
          m = fmaxf(ref[0][r], m - kLift);
          by[r] = ex2_approx(ref[0][r] - m);
          ref[0][r] = m;
          l[0][r] *= by[r];
          ofs[0][r] *= by[r];
        }
#pragma unroll
        for (int f = 0; f < FT; ++f)
#pragma unroll
          for (int z = 0; z < 4; ++z) o[0][f][z] *= by[z & 1];
      }
      const float w0 = ex2_approx(x[0] - ref[0][0]), w1 = ex2_approx(x[1] - ref[0][1]);
      fma2(l[0][0], l[0][1], w0, w1, v_inv, v_inv, l[0][0], l[0][1]);
      const uint32_t w = pack_f16x2(w0, w1);
      // (the offsets with the rounded weights, as the codes have them: what the
      // rounding does to both is relative to the value, not to its two parts)
      fma2(ofs[0][0], ofs[0][1], half_lo(w), half_hi(w), v_ofs, v_ofs, ofs[0][0], ofs[0][1]);
      // columns 2 j, 2 j + 1 of block j's keys: a column pair sums a quarter of the keys
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) pt[0][m][h] = transposed(j == 2 * m + h ? w : 0u);
    } else {
      // the keys' factors by way of shared memory: lane's own key to the lanes of its row
      const int slot = 8 * j + g;  // (row g of block j)
      __syncwarp();  // (the tile before is read)
      keys[slot] = make_float4(mine.step, mine.lo, mine.v_log, mine.v_inv);
      keys_ofs[slot] = mine.v_ofs;
      __syncwarp();
      float4 kf[MT][2];
      float v_ofs[MT][2];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          kf[m][h] = keys[16 * m + 8 * h + g];
          v_ofs[m][h] = keys_ofs[16 * m + 8 * h + g];
        }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float t0, t1, u0, u1;
            mul2(t0, t1, s[n][m][2 * h], s[n][m][2 * h + 1], fa[n][0], fa[n][1]);
            fma2(u0, u1, fb[n][0], fb[n][1], kf[m][h].y, kf[m][h].y, kf[m][h].z, kf[m][h].z);
            fma2(s[n][m][2 * h], s[n][m][2 * h + 1], t0, t1, kf[m][h].x, kf[m][h].x, u0, u1);
          }
      if (masked) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int key = key0 + 16 * m + 8 * h + key_of_row<W>(g), off = key - it.n;
            bool any = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                bool sees = key < stop;
                if (sees && off >= 0)  // (off < 256: the drafted tokens end there)
                  sees = (masks[8 * n + 2 * j + r][off >> 6] >> (off & 63)) & 1;
                if (!sees) s[n][m][2 * h + r] = -INFINITY;
                any = any || sees;
              }
            // (what hides from all of them may hold anything, and 0 * NaN would be NaN)
            if (!any) kf[m][h].w = v_ofs[m][h] = 0.f;
          }
      }
      float top = -INFINITY;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float m = fmaxf(s[n][0][r], s[n][0][2 + r]);
#pragma unroll
          for (int x = 1; x < MT; ++x) m = fmax3(m, s[n][x][r], s[n][x][2 + r]);
          top = fmaxf(top, m - ref[n][r]);
        }
      if (__any_sync(0xffffffffu, top > kLift + kSlack)) {
        // references up to this tile's maxima, what was summed down by as much
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float by[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float m = fmaxf(s[n][0][r], s[n][0][2 + r]);
#pragma unroll
            for (int x = 1; x < MT; ++x) m = fmax3(m, s[n][x][r], s[n][x][2 + r]);
#pragma unroll
            for (int z = 4; z < 32; z <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, z));
            m = fmaxf(ref[n][r], m - kLift);
            by[r] = ex2_approx(ref[n][r] - m);
            ref[n][r] = m;
            l[n][r] *= by[r];
            ofs[n][r] *= by[r];
          }
#pragma unroll
          for (int f = 0; f < FT; ++f)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[n][f][x] *= by[x & 1];
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float w0, w1;
            add2(w0, w1, s[n][m][2 * h], s[n][m][2 * h + 1], -ref[n][0], -ref[n][1]);
            w0 = ex2_approx(w0);
            w1 = ex2_approx(w1);
            fma2(l[n][0], l[n][1], w0, w1, kf[m][h].w, kf[m][h].w, l[n][0], l[n][1]);
            const uint32_t w = pack_f16x2(w0, w1);
            // (the offsets with the rounded weights, as the codes have them: what the
            // rounding does to both is relative to the value, not to its two parts)
            fma2(ofs[n][0], ofs[n][1], half_lo(w), half_hi(w), v_ofs[m][h], v_ofs[m][h], ofs[n][0], ofs[n][1]);
            pt[n][m][h] = transposed(w);
          }
    }
    // ---- o += V^T P^T
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      uint32_t vc[4][VW];
#pragma unroll
      for (int x = 0; x < 4; ++x) ld_shared<VW>(tile + v_at[x & 1] + (16 * m + 8 * (x >> 1)) * C::ROW, vc[x]);
#pragma unroll
      for (int y = 0; y < VW; ++y)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t sel = 0x4400u + 0x1111u * b;  // byte b of two keys' words
          const uint32_t x0 = __byte_perm(vc[0][y], vc[1][y], sel);
          const uint32_t x1 = __byte_perm(vc[2][y], vc[3][y], sel);
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma_f16(o[n][4 * y + b], x0 & 0x000f000fu, x0 & 0x00f000f0u, x1 & 0x000f000fu, x1 & 0x00f000f0u,
                    pt[n][m][0], pt[n][m][1]);
        }
    }
    __syncwarp();  // (every lane has read the tile)
    if (lane == 0 && key0 + C::ST * kKeys < stop) request(key0 + C::ST * kKeys, stage);
    if (++stage == C::ST) {
      stage = 0;
      parity ^= 1;
    }
  }
  if (!ok) {
    // gave up: the copies in flight must land before the CTA exits (each wait is bounded)
    volatile int never = 0;
    for (int s = 0; s < C::ST; ++s) mbar_wait(bars + 8 * s, parity ^ (s < stage ? 1 : 0), &never, p.status, 0);
  }

  // ---- the warps' sums together
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int z = FEW ? 1 : 4; z < 32; z <<= 1) {
        l[n][r] += __shfl_xor_sync(0xffffffffu, l[n][r], z);
        ofs[n][r] += __shfl_xor_sync(0xffffffffu, ofs[n][r], z);
      }
      const int row = FEW ? r : 8 * n + 2 * j + r;
      if (FEW ? lane == 0 : g == 0) {
        stats[warp][row][0] = ref[n][r];
        stats[warp][row][1] = l[n][r];
        stats[warp][row][2] = ofs[n][r];
      }
    }
  const bool whole = it.splits == 1;
  const long long first_part = static_cast<long long>(it.part - it.b) * p.T * p.H;  // (rows count from sequence 0)
  auto sums = [&](int w, int column, int at) {
    return reinterpret_cast<float*>(smem + w * C::RING) + column * C::RS + at;
  };
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (n > 0) {
      if (it.rb * NR + 8 * n >= n_rows) break;
      __syncthreads();  // (the block before is read)
    }
#pragma unroll
    for (int f = 0; f < FT; ++f)
#pragma unroll
      for (int x = 0; x < 4; ++x)  // (codes are 2^-24, odd features 2^-20)
        *sums(warp, 2 * j + (x & 1), C::GS * g + 2 * f + (x >> 1)) = o[n][f][x] * (x >> 1 ? 1048576.f : 16777216.f);
    __syncthreads();
    for (int x = static_cast<int>(threadIdx.x); x < (FEW ? 2 : 8) * (W / 2); x += 32 * kWarps) {
      const int c = x / (W / 2), r = 8 * n + c, f = 2 * (x % (W / 2));
      int t;
      const int out = out_row(r, &t);
      if (out < 0) break;  // (rows only grow)
      float m = kNoRef;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, stats[w][r][0]);
      float y0 = 0.f, y1 = 0.f, L = 0.f;
      if (t < it.live && m != kNoRef && *abort_flag == 0) {
        float add = 0.f;
        const int at = C::GS * (f / (W / 8)) + f % (W / 8);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float a = ex2_approx(stats[w][r][0] - m);
          L = fmaf(a, stats[w][r][1], L);
          add = fmaf(a, stats[w][r][2], add);
          float2 v = *reinterpret_cast<const float2*>(sums(w, c, at));
          if constexpr (FEW) {
#pragma unroll
            for (int z = 2; z < 8; z += 2) {
              const float2 u = *reinterpret_cast<const float2*>(sums(w, z + c, at));
              v.x += u.x;
              v.y += u.y;
            }
          }
          y0 = fmaf(a, v.x, y0);
          y1 = fmaf(a, v.y, y1);
        }
        y0 += add;
        y1 += add;
      }
      if (!whole) {
        if (f == 0) {
          p.part_m[first_part + out] = L == 0.f ? -INFINITY : m;
          p.part_l[first_part + out] = L;
        }
        *reinterpret_cast<float2*>(p.part_o + (first_part + out) * W + f) = make_float2(y0, y1);
        continue;
      }
      const float inv = L == 0.f ? 0.f : 1.f / L;
      if (f < p.d)
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + static_cast<long long>(out) * p.d + f) =
            pack_bf16x2(y0 * inv, y1 * inv);
      if (p.lse && f == 0)
        p.lse[(static_cast<long long>(it.b) * p.H + out % p.H) * p.T + t] =
            L == 0.f ? -INFINITY : (m + __log2f(L)) * 0.69314718055994531f;
    }
  }
}

// Calls f with the kernel's configuration for R rows per key head of d features.
template <typename F>
void with_config(int d, int R, F&& f) {
  if (d <= 64) {
    if (R <= 2) f(Q4Cfg<64, 1, true, 4, 6>{});
    else if (R <= 8) f(Q4Cfg<64, 1, false, 4, 5>{});
    else f(Q4Cfg<64, 2, false, 4, 4>{});
  } else if (d <= 128) {
    if (R <= 2) f(Q4Cfg<128, 1, true, 2, 5>{});
    else if (R <= 8) f(Q4Cfg<128, 1, false, 2, 4>{});
    else if (R <= 16) f(Q4Cfg<128, 2, false, 3, 3>{});
    else f(Q4Cfg<128, 4, false, 3, 2>{});
  } else {
    if (R <= 2) f(Q4Cfg<256, 1, true, 2, 3>{});
    else if (R <= 8) f(Q4Cfg<256, 1, false, 2, 3>{});
    else f(Q4Cfg<256, 2, false, 2, 2>{});
  }
}

template <class C>
cudaError_t launch_cfg(const RowsParams& p, cudaStream_t stream, LaunchInfo* info) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static bool attr_set[64] = {};
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(rows_q4_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  const dim3 grid(static_cast<unsigned>(p.B * p.units * p.n_splits));
  e = launch_serialized(rows_q4_kernel<C>, grid, dim3(32 * kWarps), C::SMEM, stream, p);
  if (info) {
    info->kernels = 1;
    info->grid = static_cast<int>(grid.x);
    info->block = 32 * kWarps;
    info->smem = C::SMEM;
  }
  return e;
}

}  // namespace

RowsQ4Shape rows_q4_shape(int d, int R) {
  RowsQ4Shape s = {};
  with_config(d, R, [&](auto cfg) {
    using C = decltype(cfg);
    s.width = C::W;
    s.rows = C::NR;
    s.ctas = C::CTAS;
  });
  return s;
}

cudaError_t launch_rows_q4(const RowsParams& p, cudaStream_t stream, LaunchInfo* info) {
  cudaError_t e = cudaSuccess;
  with_config(p.d, p.T * p.G, [&](auto cfg) { e = launch_cfg<decltype(cfg)>(p, stream, info); });
  return e;
}

}  // namespace mha

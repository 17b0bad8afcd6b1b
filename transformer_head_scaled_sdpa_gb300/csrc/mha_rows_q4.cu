// mha_rows_q4.cu -- attention of a few query rows per sequence over the 4-bit
// key/value cache (the decode step and the step of a tree of drafted tokens), up to
// sixteen rows per key head (32 of heads up to 64 features), sm_103a.
//
// A cached row of a key head is x = lo + step * c with codes c = 0 .. 15 (q4.cuh), so
//   s_jr = scale q_r . k_j = scale (stepk_j (q_r . c_j) + lok_j sum_f q_rf)
//   o_r  = sum_j a_jr v_j  = sum_j (a_jr stepv_j) (c_j + lov_j / stepv_j)
// and both products are of the codes alone, with a key's offset and step applied to
// its scores and weights.  The softmax keeps w_jr = 2^(s_jr + log2 stepv_j - m_r): the
// products take w, the denominator adds w / stepv, the offsets' share of the output is
// the row's sum of w lov / stepv.
//
// Codes reach the tensor core as they lie: four bits in the low bits of an fp16 are the
// subnormal c 2^-24, exact, so unpacking is a mask (one per two codes, and a shift per
// eight; the odd nibbles stay 16 times too large, and q, or the output, is divided by 16
// there).  A CTA is four warps and a ring of tiles of 128 keys and values, filled by TMA;
// a warp has 32 keys of a tile, with sums and references of its own, and the four meet
// once, at the end of the unit.  The last warp to leave a stage refills it.
//   S^T [16 keys x 8 rows] = K [16 x d] Q^T: ldmatrix gives lane (g, j) bytes 4 j .. of 16
//     of a key's row; the order of the features along the reduction is free, and Q is laid
//     out in the same one.
//   O^T [16 features x 8 rows] += V^T [16 x 16 keys] P^T: ldmatrix.trans gives a lane 16
//     bits (four features) of two keys, whose nibbles are the fragment's features.
// The weights' fragment is the scores' transposed (movmatrix).  One or two rows fill the
// eight columns with copies, so that every column pair has all the scores and each lane
// computes the weights of one key.
//
// mma.sync and not tcgen05 for these few rows: reading the cache bounds them (68 bytes per
// row of 128 features), and tcgen05 wants the codes in 8 bits or more, in shared or tensor
// memory: the packed tile written and read, the unpacked one written and read, and a CTA
// of a dozen warps that hand it on; with it, 4 x 96 heads x 16 rows take 52 us against
// 35 (8 x 48 heads x 16 rows of 64 features x 2,048 to 4,096 keys 109 against 43).  fp8 operands bring nothing here
// (mma.sync converts e4m3 to fp16 first on this machine).
//
// q is scaled by a power of two to [2^14, 2^15) at its row's largest and then exact in fp16
// to half its smallest place, 2^-25: 2^-39 of the row's largest, and 2^-35 in the odd
// features, which are divided by 16 first.  The weights are rounded to fp16 (2^-11 relative);
// products' sums (rows_q4.cuh: what they cut), the denominator and the offsets' are float32.  Weights are 2^kLift at a row's
// reference m, which moves when a tile's largest weight would pass 2^kLimit.
//
// What bounds it: 16 x 96 heads x 1,024 to 2,048 keys of 128 features, 322 MB, 61 us (5.3
// TB/s; the same launch without the arithmetic 53): 1,536 units on 608 CTAs, each of which
// waits 4 to 5 us for its lengths, Q and first tile and for its merge, and 0.46 of the
// issue slots (the masks' and shifts' pipe 0.35, the tensor pipe 0.29).  2 x 8 key heads x
// 40,001 to 65,537 keys, 4 rows: 30 us, 7 of them latency at both ends and 5 the merge of
// splits.  4 x 96 heads x 16 rows x 1,024 to 2,048 keys: 35.0 us, one wave of 384 units on
// 456 CTAs as long as its longest.  128 x 8 heads x 16 to 256 keys of 64 features: 8 us.
#include <cuda_bf16.h>

#include "rows_q4.cuh"

namespace mha {
namespace {

constexpr int kTile = 32;           // keys of a warp's part of a tile of kKeys
constexpr int kRoleRowsQ4 = 20;
// Rows per key head up to which a step is this file's.
constexpr int few_rows(int d) { return d <= 64 ? 32 : 16; }

// D += A B, 16 x 16 by 16 x 8 in fp16, ...
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// ... onto 0.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Four matrices of 8 rows x 16 bytes: lane (g, j) gets bytes 4 j .. of row g, ...
__device__ __forceinline__ void ld_rows(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
// ... or the g-th 16 bits of rows 2 j and 2 j + 1.
__device__ __forceinline__ void ld_columns16(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// A fragment of codes: the low nibbles of the halves of two words, and the next ones
// (16 times too large).
__device__ __forceinline__ void codes_of(uint32_t (&a)[4], uint32_t w0, uint32_t w1, bool across) {
  a[0] = w0 & 0x000f000fu;
  a[across ? 2 : 1] = w0 & 0x00f000f0u;
  a[across ? 1 : 2] = w1 & 0x000f000fu;
  a[3] = w1 & 0x00f000f0u;
}

// Scores of a warp's 32 keys with NQ blocks of 8 columns.  `at`: lane's address for
// ld_rows (row lane % 16, 16-byte piece lane / 16), frag(i, x): Q's fragment of reduction
// step i and column block x.  (A product waits some 27 cycles for the one before on the
// same sums, so there are four or more sums to take turns: two blocks of keys, and of one
// block of columns the even and odd steps apart.)
template <int W, int NQ, typename F>
__device__ __forceinline__ void score_products(uint32_t at, float (&s)[2][NQ][4], F&& frag) {
  constexpr int PARTS = NQ == 1 ? 2 : 1;
  float part[2][4];
#pragma unroll
  for (int c = 0; c < W / 32; c += 2) {
    uint32_t w[2][4];
#pragma unroll
    for (int m = 0; m < 2; ++m) ld_rows((at + 16 * m * (W / 2)) ^ (16 * c), w[m]);
#pragma unroll
    for (int z = 0; z < 4; ++z) {
      uint32_t a[2][4];
#pragma unroll
      for (int m = 0; m < 2; ++m)
        codes_of(a[m], z & 1 ? w[m][z & 2] >> 8 : w[m][z & 2], z & 1 ? w[m][(z & 2) + 1] >> 8 : w[m][(z & 2) + 1], true);
#pragma unroll
      for (int x = 0; x < NQ; ++x) {
        const uint2 b = frag(2 * c + z, x);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          float(&y)[4] = PARTS == 2 && (z & 1) ? part[m] : s[m][x];
          if (c == 0 && z < PARTS) mma_f16_first(y, a[m], b.x, b.y);
          else mma_f16(y, a[m], b.x, b.y);
        }
      }
    }
  }
  if constexpr (PARTS == 2) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[m][0][i] += part[m][i];
  }
}

// A row's fragments of Q: lane (g, j) has the features 32 c + 8 j .. + 7 (v[c]) of its
// column's row; put(i, b) gets the fragment of reduction step i.  Returns the e of its
// factor 2^e and its sum (every lane of the column's).
struct QRow {
  int e;
  float sum;
};
template <int KC, typename F>
__device__ __forceinline__ QRow q_fragments(const uint4 (&v)[KC], F&& put) {
  float amax = 0.f;
#pragma unroll
  for (int c = 0; c < KC; ++c) {
    const uint32_t x[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
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
  for (int c = 0; c < KC; ++c) {
    const float y[8] = {bf16_lo(v[c].x) * inv, bf16_hi(v[c].x) * inv, bf16_lo(v[c].y) * inv, bf16_hi(v[c].y) * inv,
                        bf16_lo(v[c].z) * inv, bf16_hi(v[c].z) * inv, bf16_lo(v[c].w) * inv, bf16_hi(v[c].w) * inv};
#pragma unroll
    for (int x = 0; x < 8; ++x) sum += y[x];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      put(2 * c + h, make_uint2(pack_f16x2(y[2 * h], y[4 + 2 * h]),
                                pack_f16x2(y[2 * h + 1] * 0.0625f, y[5 + 2 * h] * 0.0625f)));
  }
  sum += __shfl_xor_sync(0xffffffffu, sum, 1);
  sum += __shfl_xor_sync(0xffffffffu, sum, 2);
  return {e, sum};
}

// Adds one to a count in shared memory, behind what the warp read and ahead of what it
// does next; returns the count before.
__device__ __forceinline__ uint32_t arrive_count(uint32_t at) {
  uint32_t n;
  asm volatile("atom.acq_rel.cta.shared::cta.add.u32 %0, [%1], 1;" : "=r"(n) : "r"(at) : "memory");
  return n;
}

// ---------------------------------------------------------------------------
// W: widest head; ROWS: 1, 2 or a multiple of 8; ST: stages of the ring; CTAS: per SM.
// ---------------------------------------------------------------------------
template <int W_, int ROWS_, int ST_, int CTAS_>
struct Q4Cfg {
  static constexpr int W = W_, NR = ROWS_, ST = ST_, CTAS = CTAS_;
  static constexpr int WP = 4;
  static constexpr bool FEW = NR <= 2;
  static constexpr int NT = FEW ? 1 : NR / 8;      // blocks of 8 columns
  static constexpr int ROW = W / 2;                // bytes of a tile's row
  static constexpr int KC = W / 32;                // 16-byte pieces of a row: 32 features
  static constexpr int FT = W / 16;                // blocks of 16 features
  static constexpr bool Q_SHARED = KC * NT > 4;    // Q's fragments in shared memory
  static constexpr int RS = W + 4;                 // merge: floats of a warp's column of sums (16-byte stores hit all banks)
  static constexpr int TILE = kKeys * ROW;         // bytes of a tile's keys, and of its values
  static constexpr int SUMS = 8 * NT * RS * 4;     // a warp's, in the ring at the end
  static constexpr int RING = ST * 2 * TILE;
  static_assert(RING >= WP * SUMS, "ring");
  static constexpr int OFF_BAR = RING;             // barriers [stage], warps that left it [stage]
  static constexpr int OFF_ABORT = OFF_BAR + ST * 12;
  static constexpr int OFF_MASKS = (OFF_ABORT + 4 + 15) / 16 * 16;  // uint64 [NR][4]
  static constexpr int OFF_STATS = OFF_MASKS + NR * 32;             // float [warp][NR][3]
  static constexpr int OFF_SCALES = (OFF_STATS + WP * NR * 12 + 15) / 16 * 16;
  static constexpr int OFF_KEYS = OFF_SCALES + Scales::BYTES;  // float4 [warp][32], float [warp][32]
  static constexpr int OFF_Q = OFF_KEYS + (FEW ? 0 : WP * kTile * 20);        // uint2 [2 KC NT][32]
  static constexpr int SMEM = OFF_Q + (Q_SHARED ? 2 * KC * NT * 256 : 0) + 1024;
};

template <class C>
__global__ void __launch_bounds__(32 * C::WP, C::CTAS) rows_q4_kernel(const __grid_constant__ RowsParams p) {
  constexpr int W = C::W, NT = C::NT, KC = C::KC, FT = C::FT, NR = C::NR;
  constexpr bool FEW = C::FEW;
  constexpr int MT = kTile / 16;
  constexpr int LANE_ROWS = NR == 1 ? 1 : 2;  // rows of a lane's scores
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
  uint64_t(*masks)[4] = reinterpret_cast<uint64_t(*)[4]>(smem + C::OFF_MASKS);
  float(*stats)[NR][3] = reinterpret_cast<float(*)[NR][3]>(smem + C::OFF_STATS);
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int g = lane >> 2, j = lane & 3;
  const uint32_t ring = smem_u32(smem), full = ring + C::OFF_BAR, left = full + 8 * C::ST;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::ST; ++s) {
      mbar_init(full + 8 * s, 1);
      reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 8 * C::ST)[s] = 0;
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  griddep_wait();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int n_rows = p.T * p.G;
  Unit it;
  if (!this_unit(p, (n_rows + NR - 1) / NR, kSms * C::CTAS, lane, &it)) return;

  const int stop = min(it.t1 * kKeys, it.end), first = it.t0 * kKeys;
  const Loader<W> load{p, it, stop};
  // Output row of row r of the unit (-1 past the last), t: its drafted token.
  auto out_row = [&](int r, int* t) {
    const int gr = it.rb * NR + r;
    *t = -1;
    if (gr >= n_rows) return -1;
    *t = p.G == 1 ? gr : gr / p.G;
    return (it.b * p.T + *t) * p.H + it.hk * p.G + (gr - *t * p.G);
  };
  // Plain loads first, all of them together: behind the ring's copies each would wait
  // for several tiles.  The offsets and steps (FEW: lane (g, j) owns key g of block j of
  // 8; else key `lane`) ...
  const long long scales = (static_cast<long long>(it.b) * p.H_kv + it.hk) * p.Lk;
  const int own = kTile * warp + (FEW ? 8 * j + g : lane);
  const Scales words{ring + C::OFF_SCALES + 8 * threadIdx.x, reinterpret_cast<const uint32_t*>(p.k_scale) + scales,
                     reinterpret_cast<const uint32_t*>(p.v_scale) + scales, own, stop};
  words.start(first);
  // ... Q: lane (g, j) holds the features 32 c + 8 j .. of the row of column g of each block
  // of columns (FEW: the even columns are row 0, the odd ones row 1) ...
  uint4 v[NT][KC];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    int t;
    const int out = out_row(NR == 1 ? 0 : (NR == 2 ? g & 1 : 8 * n + g), &t);
    const bool live = out >= 0 && t < it.live;
    const uint16_t* src = static_cast<const uint16_t*>(p.q) + static_cast<long long>(max(out, 0)) * p.d;
#pragma unroll
    for (int c = 0; c < KC; ++c) {
      v[n][c] = make_uint4(0, 0, 0, 0);
      if (live && 32 * c < p.d) v[n][c] = __ldg(reinterpret_cast<const uint4*>(src + 32 * c + 8 * j));
    }
  }
  // ... and the rows' masks
  static_assert(NR * 4 <= 32 * C::WP, "a word to a thread");
  const uint64_t bits = threadIdx.x < NR * 4 ? mask_word(p, it, static_cast<int>(threadIdx.x), out_row) : 0;
  if (threadIdx.x == 0)
    for (int s = 0; s < C::ST; ++s)
      if (first + s * kKeys < stop) load(ring + s * 2 * C::TILE, full + 8 * s, first + s * kKeys);

  uint2 q[C::Q_SHARED ? 1 : 2 * KC * NT];
  uint2* q_shared = reinterpret_cast<uint2*>(smem + C::OFF_Q) + lane;
  QRow rows[NT];
  int top_e = -200;  // of the unit's rows; an infinite one, whose scores are none, has 114
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    rows[n] = q_fragments<KC>(v[n], [&](int i, uint2 b) {
      if constexpr (C::Q_SHARED) {
        if (warp == 0) q_shared[(i * NT + n) * 32] = b;
      } else {
        q[i * NT + n] = b;
      }
    });
    if (rows[n].e < 114) top_e = max(top_e, rows[n].e);
  }
  const int shift = factor_shift(__reduce_max_sync(0xffffffffu, top_e), p.scale_log2);
  const float key_scale = pow2i(shift);
  float fa[NT][2], fb[NT][2];  // factors of a row's product and of its sum: columns 8 n + 2 j, + 1
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float f = pow2i(rows[n].e) * pow2i(-shift) * p.scale_log2;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      fa[n][r] = __shfl_sync(0xffffffffu, f * 16777216.f, 8 * j + 4 * r);  // (codes are 2^-24)
      fb[n][r] = __shfl_sync(0xffffffffu, f * rows[n].sum, 8 * j + 4 * r);
    }
  }
  if (threadIdx.x < NR * 4) masks[threadIdx.x >> 2][threadIdx.x & 3] = bits;
  __syncthreads();  // (the barriers are set up, too)

  float o[NT][FT][4];
  float ref[NT][2], l[NT][2], ofs[NT][2];  // references less kLift; sums of weights, of the offsets' shares
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
  // lane's row and piece of the warp's part of a tile, for ldmatrix
  const int row16 = lane & 15;
  const uint32_t at = (kTile * warp + row16) * C::ROW + 16 * (swizzle<W>(row16) ^ (lane >> 4));
  float4* keys = reinterpret_cast<float4*>(smem + C::OFF_KEYS) + warp * kTile;
  float* keys_ofs = reinterpret_cast<float*>(smem + C::OFF_KEYS + C::WP * kTile * 16) + warp * kTile;

  bool ok = true;
  int stage = 0, i = 0;
  uint32_t parity = 0;
#pragma unroll 1
  for (int tile0 = first; tile0 < stop; tile0 += kKeys, ++i) {
    const uint32_t tile = ring + stage * 2 * C::TILE;
    const uint2 kv = words.get(i, tile0);
    KeyFactors mine = key_factors(kv.x, kv.y, key_scale);
    if constexpr (!FEW) {
      // the keys' factors by way of shared memory: lane's own key to the lanes of its row
      __syncwarp();  // (the tile before is read)
      keys[lane] = make_float4(mine.step, mine.lo, mine.v_log, mine.v_inv);
      keys_ofs[lane] = mine.v_ofs;
      __syncwarp();  // (read by the other lanes: the vote below orders no memory among them)
    }
    ok = __all_sync(0xffffffffu, mbar_wait(full + 8 * stage, parity, abort_flag, p.status, kRoleRowsQ4 * 64 + stage));
    if (!ok) break;
    const int key0 = tile0 + kTile * warp;
    if (key0 < stop) {
      // ---- scores: s[m][n] = keys g, 8 + g of block m of 16, columns 2 j, 2 j + 1 of block n
      float s[MT][NT][4];
      score_products<W, NT>(tile + at, s, [&](int i, int n) {
        if constexpr (C::Q_SHARED) return q_shared[(i * NT + n) * 32];
        else return q[i * NT + n];
      });
      // ---- weights
      const bool masked = key0 + kTile > min(it.n, stop);
      uint32_t pt[MT][NT][2];  // weights transposed: column g, keys 2 j, 2 j + 1 (+ 8)
      if constexpr (FEW) {
        // every column pair has all the keys' scores: lane (g, j) takes those of its own key
        float x[LANE_ROWS], top = -INFINITY;
#pragma unroll
        for (int r = 0; r < LANE_ROWS; ++r) {
          const float lo = j & 1 ? s[0][0][2 + r] : s[0][0][r], hi = j & 1 ? s[1][0][2 + r] : s[1][0][r];
          x[r] = fmaf((j & 2 ? hi : lo) * fa[0][r], mine.step, fmaf(fb[0][r], mine.lo, mine.v_log));
        }
        if (masked) {
          const int key = tile0 + own, off = key - it.n;
          bool any = false;
#pragma unroll
          for (int r = 0; r < LANE_ROWS; ++r) {
            bool sees = key < stop;
            if (sees && off >= 0) sees = (masks[r][off >> 6] >> (off & 63)) & 1;  // (off < 256: drafted tokens end there)
            if (!sees) x[r] = -INFINITY;
            any = any || sees;
          }
          // (of a key that hides from both: its factors are finite, see key_factors, and meet the weight
          // 0; without this line the tests above become branches: up to 2 % with 2 to 16 rows)
          if (!any) mine.v_inv = mine.v_ofs = 0.f;
        }
#pragma unroll
        for (int r = 0; r < LANE_ROWS; ++r) top = fmaxf(top, x[r] - ref[0][r]);
        if (__any_sync(0xffffffffu, top > kLimit)) {
          // references up to this tile's maxima, what was summed down by as much
          float by[2] = {1.f, 1.f};
#pragma unroll
          for (int r = 0; r < LANE_ROWS; ++r) {
            float m = x[r];
#pragma unroll
            for (int z = 1; z < 32; z <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, z));
            m = fmaxf(ref[0][r], lifted(m));
            by[r] = ex2_approx(ref[0][r] - m);
            ref[0][r] = m;
            l[0][r] *= by[r];
            ofs[0][r] *= by[r];
          }
#pragma unroll
          for (int f = 0; f < FT; ++f)
#pragma unroll
            for (int z = 0; z < 4; ++z) o[0][f][z] *= by[NR == 1 ? 0 : z & 1];
        }
        uint32_t w;
        if constexpr (NR == 1) {
          const float w0 = ex2_approx(x[0] - ref[0][0]);
          l[0][0] = fmaf(w0, mine.v_inv, l[0][0]);
          w = pack_f16x2(w0, 0.f);
          // (the offsets with the rounded weights, as the codes have them: what the
          // rounding does to both is relative to the value, not to its two parts)
          ofs[0][0] = fmaf(half_lo(w), mine.v_ofs, ofs[0][0]);
        } else {
          const float w0 = ex2_approx(x[0] - ref[0][0]), w1 = ex2_approx(x[1] - ref[0][1]);
          fma2(l[0][0], l[0][1], w0, w1, mine.v_inv, mine.v_inv, l[0][0], l[0][1]);
          w = pack_f16x2(w0, w1);
          fma2(ofs[0][0], ofs[0][1], half_lo(w), half_hi(w), mine.v_ofs, mine.v_ofs, ofs[0][0], ofs[0][1]);
        }
        // columns 2 j, 2 j + 1 of block j's keys: a column pair sums a quarter of the keys
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) pt[m][0][h] = transposed(j == 2 * m + h ? w : 0u);
      } else {
        float v_inv[MT][2], v_ofs[MT][2];
        float top = -INFINITY;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float4 kf = keys[16 * m + 8 * h + g];
            v_inv[m][h] = kf.w;
            v_ofs[m][h] = keys_ofs[16 * m + 8 * h + g];
            bool any = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float* y = s[m][n] + 2 * h;
              float t0, t1, u0, u1;
              mul2(t0, t1, y[0], y[1], fa[n][0], fa[n][1]);
              fma2(u0, u1, fb[n][0], fb[n][1], kf.y, kf.y, kf.z, kf.z);
              fma2(y[0], y[1], t0, t1, kf.x, kf.x, u0, u1);
            }
            if (masked) {
              const int key = key0 + 16 * m + 8 * h + g, off = key - it.n;
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  bool sees = key < stop;
                  if (sees && off >= 0)  // (off < 256: the drafted tokens end there)
                    sees = (masks[8 * n + 2 * j + r][off >> 6] >> (off & 63)) & 1;
                  if (!sees) s[m][n][2 * h + r] = -INFINITY;
                  any = any || sees;
                }
              // (as above)
              if (!any) v_inv[m][h] = v_ofs[m][h] = 0.f;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) top = fmax3(top, s[m][n][2 * h] - ref[n][0], s[m][n][2 * h + 1] - ref[n][1]);
          }
        if (__any_sync(0xffffffffu, top > kLimit)) {
          // references up to this tile's maxima, what was summed down by as much
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float by[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float m = fmaxf(s[0][n][r], s[0][n][2 + r]);
#pragma unroll
              for (int x = 1; x < MT; ++x) m = fmax3(m, s[x][n][r], s[x][n][2 + r]);
#pragma unroll
              for (int z = 4; z < 32; z <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, z));
              m = fmaxf(ref[n][r], lifted(m));
              by[r] = ex2_approx(ref[n][r] - m);
              ref[n][r] = m;
              l[n][r] *= by[r];
              ofs[n][r] *= by[r];
            }
#pragma unroll
            for (int f = 0; f < FT; ++f)
#pragma unroll
              for (int z = 0; z < 4; ++z) o[n][f][z] *= by[z & 1];
          }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float w0, w1;
              add2(w0, w1, s[m][n][2 * h], s[m][n][2 * h + 1], -ref[n][0], -ref[n][1]);
              w0 = ex2_approx(w0);
              w1 = ex2_approx(w1);
              fma2(l[n][0], l[n][1], w0, w1, v_inv[m][h], v_inv[m][h], l[n][0], l[n][1]);
              const uint32_t w = pack_f16x2(w0, w1);
              // (the offsets with the rounded weights, as above)
              fma2(ofs[n][0], ofs[n][1], half_lo(w), half_hi(w), v_ofs[m][h], v_ofs[m][h], ofs[n][0], ofs[n][1]);
              pt[m][n][h] = transposed(w);
            }
      }
      // ---- o += V^T P^T, 16 keys at a time
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < KC; c += 2) {
          uint32_t w[4];
          ld_columns16((tile + C::TILE + 16 * m * C::ROW + at) ^ (16 * c), w);
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            uint32_t a[4];
            codes_of(a, z & 1 ? w[z & 2] >> 8 : w[z & 2], z & 1 ? w[(z & 2) + 1] >> 8 : w[(z & 2) + 1], false);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(o[n][2 * c + z], a, pt[m][n][0], pt[m][n][1]);
          }
        }
      __syncwarp();  // (every lane has read the tile)
    }
    // the last warp to leave a stage fills it again
    if (lane == 0 && arrive_count(left + 4 * stage) % C::WP == C::WP - 1 && tile0 + C::ST * kKeys < stop)
      load(tile, full + 8 * stage, tile0 + C::ST * kKeys);
    __syncwarp();
    if (++stage == C::ST) {
      stage = 0;
      parity ^= 1;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");  // (gave up: offsets and steps, too, are in flight)
  __syncthreads();
  if (*abort_flag != 0 && threadIdx.x == 0) {
    // gave up: the copies in flight must land before the CTA exits (each wait is bounded)
    volatile int never = 0;
    for (int s = 0; s < C::ST; ++s) {
      mbar_wait(full + 8 * s, 0, &never, p.status, 0);
      mbar_wait(full + 8 * s, 1, &never, p.status, 0);
    }
  }

  // ---- the warps' sums together
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int r = 0; r < LANE_ROWS; ++r) {
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
    return reinterpret_cast<float*>(smem + w * C::SUMS) + column * C::RS + at;
  };
  // (four features of a piece, 4 g .. + 3, of the two columns of each block)
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < KC; ++c)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        *reinterpret_cast<float4*>(sums(warp, 8 * n + 2 * j + r, 32 * c + 4 * g)) =
            make_float4(o[n][2 * c][r], o[n][2 * c][2 + r], o[n][2 * c + 1][r], o[n][2 * c + 1][2 + r]);
  __syncthreads();
  // (a row to a warp: once per unit, so short code counts)
#pragma unroll 1
  for (int r = warp; r < NR; r += C::WP) {
    int t;
    const int out = out_row(r, &t);
    if (out < 0) break;
    float m = kNoRef;
#pragma unroll
    for (int w = 0; w < C::WP; ++w) m = fmaxf(m, stats[w][r][0]);
    float a[C::WP], L = 0.f, add = 0.f;
    // (a row that saw no key has sums of 0; one whose scores are all NaN has NaN, and shows it)
    const bool live = t < it.live && *abort_flag == 0;
#pragma unroll
    for (int w = 0; w < C::WP; ++w) {
      a[w] = live ? ex2_approx(stats[w][r][0] - m) : 0.f;
      if (live) {
        L = fmaf(a[w], stats[w][r][1], L);
        add = fmaf(a[w], stats[w][r][2], add);
      }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    if (lane == 0) {
      if (!whole) {
        p.part_m[first_part + out] = L == 0.f ? -INFINITY : m;
        p.part_l[first_part + out] = L;
      } else if (p.lse) {
        p.lse[(static_cast<long long>(it.b) * p.H + out % p.H) * p.T + t] =
            L == 0.f ? -INFINITY : (m + __log2f(L)) * 0.69314718055994531f;
      }
    }
#pragma unroll 1
    for (int f = 2 * lane; f < W; f += 64) {
      float y0 = 0.f, y1 = 0.f;
#pragma unroll
      for (int w = 0; w < C::WP; ++w) {
#pragma unroll
        for (int z = 0; z < (FEW ? 8 : 1); z += 2) {
          const float2 u = *reinterpret_cast<const float2*>(sums(w, z + r, f));
          y0 = fmaf(a[w], u.x, y0);
          y1 = fmaf(a[w], u.y, y1);
        }
      }
      // (codes are 2^-24, odd features' 2^-20; what is not live may be anything)
      y0 = live ? fmaf(y0, 16777216.f, add) : 0.f;
      y1 = live ? fmaf(y1, 1048576.f, add) : 0.f;
      if (!whole)
        *reinterpret_cast<float2*>(p.part_o + (first_part + out) * W + f) = make_float2(y0, y1);
      else if (f < p.d)
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + static_cast<long long>(out) * p.d + f) =
            pack_bf16x2(y0 * inv, y1 * inv);
    }
  }
}

// Calls f with the kernel's configuration for R rows per key head of d features.  us over
// 8 sequences of 2,048 to 4,096 keys, 48 heads of 64 features, 24 of 128 or 12 of 256:
// as here, in a unit for twice the rows or more, and in units for fewer:
//   rows     64                 128               256
//    1       28.4  29.5         22.6 23.3         23.4 23.6
//    2       29.8  30.3 52.6    23.7 25.2 43.2    23.6 25.0 39.5
//    8       31.4  41.5 73.3    25.9 38.6 62.7    26.4 31.6 60.0
//   16       42.6 109.2 50.9    39.8 47.6 49.8    33.0 51.9 51.8   (wider: the other kernel)
//   32       66.5 110.4         48.9      60.0    52.6      68.7   (128, 256: the other kernel)
// Stages and CTAs to an SM were swept with them.  More CTAs hide the ends of units, more
// stages the memory: one row of 64 features over 128 x 8 heads x 16 to 256 keys 8.0 us with
// seven CTAs of three stages, 10.6 with six of four, 9.8 with ten of two; eight rows of 64
// 31.3 with five CTAs of two stages, 37.6 with four of four; of 256 26.4 with two CTAs of
// three stages, 32.5 with three of two.
template <typename F>
void with_config(int d, int R, F&& f) {
  if (d <= 64) {
    if (R == 1) f(Q4Cfg<64, 1, 3, 7>{});
    else if (R == 2) f(Q4Cfg<64, 2, 3, 7>{});
    else if (R <= 8) f(Q4Cfg<64, 8, 2, 5>{});
    else f(Q4Cfg<64, 16, 4, 3>{});
  } else if (d <= 128) {
    if (R == 1) f(Q4Cfg<128, 1, 3, 4>{});
    else if (R == 2) f(Q4Cfg<128, 2, 3, 4>{});
    else if (R <= 8) f(Q4Cfg<128, 8, 2, 4>{});
    else f(Q4Cfg<128, 16, 3, 3>{});
  } else {
    if (R == 1) f(Q4Cfg<256, 1, 2, 3>{});
    else if (R == 2) f(Q4Cfg<256, 2, 2, 3>{});
    else if (R <= 8) f(Q4Cfg<256, 8, 3, 2>{});
    else f(Q4Cfg<256, 16, 3, 2>{});
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
  e = launch_serialized(rows_q4_kernel<C>, grid, dim3(32 * C::WP), C::SMEM, stream, p);
  if (info) {
    info->kernels = 1;
    info->grid = static_cast<int>(grid.x);
    info->block = 32 * C::WP;
    info->smem = C::SMEM;
  }
  return e;
}

}  // namespace

RowsQ4Shape rows_q4_shape(int d, int R) {
  if (R > few_rows(d)) return rows_q4_many_shape(d, R);
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
  if (p.T * p.G > few_rows(p.d)) return launch_rows_q4_many(p, stream, info);
  cudaError_t e = cudaSuccess;
  with_config(p.d, p.T * p.G, [&](auto cfg) { e = launch_cfg<decltype(cfg)>(p, stream, info); });
  return e;
}

}  // namespace mha

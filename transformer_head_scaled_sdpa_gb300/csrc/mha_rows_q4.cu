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
constexpr float kLift = 8.f;    // weights are 2^kLift at their reference
constexpr float kSlack = 7.f;   // and stay below 2^(kLift + kSlack), inside fp16's range
constexpr float kNoRef = -3.0e38f;  // a row that has seen no key

template <int W_, int NT_, int KT_, int CTAS_>
struct Q4Cfg {
  static constexpr int W = W_;        // widest head
  static constexpr int NT = NT_;      // blocks of 8 rows
  static constexpr int KT = KT_;      // keys a warp has in registers
  static constexpr int CTAS = CTAS_;  // per SM
  static constexpr int NR = 8 * NT;
  static constexpr int MT = KT / 16;  // blocks of 16 keys
  static constexpr int KW = W / 32;   // words of a key's row per lane
  static constexpr int VW = W / 64;   // words of a value's row per lane
  static constexpr int FT = W / 16;   // blocks of 16 features
  static constexpr bool Q_SHARED = W * NT > 128;  // Q's fragments in shared memory
  // merge: a warp's row of sums, eight lanes' features 4 floats apart
  static constexpr int GS = W / 8 + 4;
  static constexpr int RS = 8 * GS + 2;
};

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

// N consecutive words (N * 4-byte aligned up to 16).
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* at, uint32_t* w) {
  if constexpr (N == 1) {
    w[0] = __ldg(reinterpret_cast<const uint32_t*>(at));
  } else if constexpr (N == 2) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(at));
    w[0] = v.x, w[1] = v.y;
  } else {
    static_assert(N == 4, "words");
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(at));
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
}

template <class C>
__global__ void __launch_bounds__(32 * kWarps, C::CTAS) rows_q4_kernel(const __grid_constant__ RowsParams p) {
  constexpr int W = C::W, NT = C::NT, KT = C::KT, MT = C::MT, KW = C::KW, VW = C::VW, FT = C::FT, NR = C::NR;
  __shared__ __align__(16) float sums[kWarps][NR][C::RS];   // O of each warp
  __shared__ float stats[kWarps][NR][3];                    // m, l and the offsets' sum
  __shared__ uint64_t masks[NR][4];
  __shared__ uint2 q_frags[C::Q_SHARED ? 2 * KW * NT : 1][32];
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int g = lane >> 2, j = lane & 3;
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
  // Output row of row r of the unit (-1 past the last), t: its drafted token.
  auto out_row = [&](int r, int* t) {
    const int gr = it.rb * NR + r;
    *t = -1;
    if (gr >= n_rows) return -1;
    *t = p.G == 1 ? gr : gr / p.G;
    return (it.b * p.T + *t) * p.H + it.hk * p.G + (gr - *t * p.G);
  };

  const int stop = min(it.t1 * kKeys, it.end);  // keys first .. stop - 1 are the unit's
  const long long pitch = static_cast<long long>(p.H_kv) * (p.d / 2);  // bytes between positions
  const int key_bytes = static_cast<int>(pitch);
  const long long base = static_cast<long long>(it.b) * p.Lk * pitch + static_cast<long long>(it.hk) * (p.d / 2);
  // lane's part of a key's row: bytes 4 KW j (16 j and 64 + 16 j when 256 wide), of a value's: 4 VW g
  constexpr int KV = KW > 4 ? 4 : KW;  // words loaded at once
  const uint8_t* k_at = static_cast<const uint8_t*>(p.k_codes) + base + 4 * KV * j;
  const uint8_t* v_at = static_cast<const uint8_t*>(p.v_codes) + base + 4 * VW * g;
  const bool k_has[2] = {8 * KV * j < p.d, 128 + 8 * KV * j < p.d};
  const bool v_has = 8 * VW * g < p.d;  // (d is a multiple of 32: a lane's part is inside the row or past it)
  const long long scales = (static_cast<long long>(it.b) * p.H_kv + it.hk) * p.Lk;
  const uint32_t* k_scale = reinterpret_cast<const uint32_t*>(p.k_scale) + scales;
  const uint32_t* v_scale = reinterpret_cast<const uint32_t*>(p.v_scale) + scales;

  uint32_t kc[MT][2][KW], vc[MT][4][VW], ks[MT][2], vs[MT][2];
  // (keys past the end are the last one again: their weight is 0)
  auto load_k = [&](int key0) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int key = min(key0 + 16 * m + 8 * h + g, stop - 1);
        const uint8_t* at = k_at + static_cast<long long>(key) * key_bytes;
#pragma unroll
        for (int w = 0; w < KW; w += KV) {
#pragma unroll
          for (int x = 0; x < KV; ++x) kc[m][h][w + x] = 0;
          if (k_has[w / KV]) load_words<KV>(at + 16 * w, kc[m][h] + w);
        }
        ks[m][h] = __ldg(k_scale + key);
        vs[m][h] = __ldg(v_scale + key);
      }
  };
  auto load_v = [&](int key0) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int key = min(key0 + 16 * m + 2 * j + (x & 1) + 8 * (x >> 1), stop - 1);
#pragma unroll
        for (int y = 0; y < VW; ++y) vc[m][x][y] = 0;
        if (v_has) load_words<VW>(v_at + static_cast<long long>(key) * key_bytes, vc[m][x]);
      }
  };
  int key0 = it.t0 * kKeys + warp * KT;
  if (key0 < stop) {
    load_k(key0);
    load_v(key0);
  }

  // ---- Q: lane (g, j) holds the features of its part of the keys' rows, of rows 8 n + g
  uint2 q[C::Q_SHARED ? 1 : 2 * KW * NT];
  float fa[NT][2], fb[NT][2];  // factors of a row's product and of its sum: rows 8 n + 2 j, + 1
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    int t;
    const int out = out_row(8 * n + g, &t);
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
          if (warp == 0) q_frags[(2 * w + h) * NT + n][lane] = b;
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
      fa[n][r] = __shfl_sync(0xffffffffu, f * 16777216.f, 8 * j + 4 * r);
      fb[n][r] = __shfl_sync(0xffffffffu, f * sum, 8 * j + 4 * r);
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
  float ref[NT][2], l[NT][2], ofs[NT][2];
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

#pragma unroll 1
  for (; key0 < stop; key0 += kWarps * KT) {
    const int next = key0 + kWarps * KT;
    // ---- scores: s[n][m] = keys g (+ 8) of block m, rows 2 j, 2 j + 1 of block n
    float s[NT][MT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[n][m][x] = 0.f;
#pragma unroll
    for (int w = 0; w < KW; ++w)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint2 b[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if constexpr (C::Q_SHARED) b[n] = q_frags[(2 * w + h) * NT + n][lane];
          else b[n] = q[(2 * w + h) * NT + n];
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const uint32_t x0 = h ? kc[m][0][w] >> 8 : kc[m][0][w], x1 = h ? kc[m][1][w] >> 8 : kc[m][1][w];
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma_f16(s[n][m], x0 & 0x000f000fu, x1 & 0x000f000fu, x0 & 0x00f000f0u, x1 & 0x00f000f0u, b[n].x, b[n].y);
        }
      }
    // a key's factor, offset, and (log2 of) its value's step
    float k_lo[MT][2], k_step[MT][2], v_log[MT][2], v_inv[MT][2], v_ofs[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        k_lo[m][h] = bf16_lo(ks[m][h]);
        k_step[m][h] = bf16_hi(ks[m][h]);
        const float step = bf16_hi(vs[m][h]);
        v_log[m][h] = lg2_approx(step);
        v_inv[m][h] = __frcp_rn(step);
        v_ofs[m][h] = bf16_lo(vs[m][h]) * v_inv[m][h];
      }
    if (next < stop) load_k(next);
    // ---- weights
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int h = x >> 1, r = x & 1;
          s[n][m][x] = fmaf(s[n][m][x] * fa[n][r], k_step[m][h], fmaf(fb[n][r], k_lo[m][h], v_log[m][h]));
        }
    const bool masked = key0 + KT > min(it.n, stop);
    if (masked) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = key0 + 16 * m + 8 * h + g, off = key - it.n;
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
          if (!any) v_inv[m][h] = v_ofs[m][h] = 0.f;
        }
    }
    float top = -INFINITY;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) top = fmax3(top, s[n][m][r] - ref[n][r], s[n][m][2 + r] - ref[n][r]);
    if (__any_sync(0xffffffffu, top > kSlack)) {
      // references up to this tile's maxima, what was summed down by as much
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float by[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float m = ref[n][r];
#pragma unroll
          for (int x = 0; x < MT; ++x) m = fmax3(m, s[n][x][r], s[n][x][2 + r]);
#pragma unroll
          for (int z = 4; z < 32; z <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, z));
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
    uint32_t pt[NT][MT][2];  // weights transposed: row g, keys 2 j, 2 j + 1 (+ 8)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float w0 = ex2_approx(s[n][m][2 * h] - ref[n][0] + kLift);
          const float w1 = ex2_approx(s[n][m][2 * h + 1] - ref[n][1] + kLift);
          l[n][0] = fmaf(w0, v_inv[m][h], l[n][0]);
          l[n][1] = fmaf(w1, v_inv[m][h], l[n][1]);
          const uint32_t w = pack_f16x2(w0, w1);
          // (the offsets with the rounded weights, as the codes have them: what the
          // rounding does to both is relative to the value, not to its two parts)
          ofs[n][0] = fmaf(half_lo(w), v_ofs[m][h], ofs[n][0]);
          ofs[n][1] = fmaf(half_hi(w), v_ofs[m][h], ofs[n][1]);
          pt[n][m][h] = transposed(w);
        }
    // ---- o += V^T P^T
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int y = 0; y < VW; ++y)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t sel = 0x4400u + 0x1111u * b;  // byte b of two keys' words
          const uint32_t x0 = __byte_perm(vc[m][0][y], vc[m][1][y], sel);
          const uint32_t x1 = __byte_perm(vc[m][2][y], vc[m][3][y], sel);
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma_f16(o[n][4 * y + b], x0 & 0x000f000fu, x0 & 0x00f000f0u, x1 & 0x000f000fu, x1 & 0x00f000f0u,
                    pt[n][m][0], pt[n][m][1]);
        }
    if (next < stop) load_v(next);
  }

  // ---- the warps' sums together
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int z = 4; z < 32; z <<= 1) {
        l[n][r] += __shfl_xor_sync(0xffffffffu, l[n][r], z);
        ofs[n][r] += __shfl_xor_sync(0xffffffffu, ofs[n][r], z);
      }
      if (g == 0) {
        stats[warp][8 * n + 2 * j + r][0] = ref[n][r];
        stats[warp][8 * n + 2 * j + r][1] = l[n][r];
        stats[warp][8 * n + 2 * j + r][2] = ofs[n][r];
      }
    }
#pragma unroll
    for (int f = 0; f < FT; ++f)
#pragma unroll
      for (int x = 0; x < 4; ++x)  // (codes are 2^-24, odd features 2^-20)
        sums[warp][8 * n + 2 * j + (x & 1)][C::GS * g + 2 * f + (x >> 1)] =
            o[n][f][x] * (x >> 1 ? 1048576.f : 16777216.f);
  }
  __syncthreads();
  const bool whole = it.splits == 1;
  const long long first_part = static_cast<long long>(it.part - it.b) * p.T * p.H;  // (rows count from sequence 0)
  for (int x = static_cast<int>(threadIdx.x); x < NR * (W / 2); x += 32 * kWarps) {
    const int r = x / (W / 2), f = 2 * (x % (W / 2));
    int t;
    const int out = out_row(r, &t);
    if (out < 0) break;  // (rows only grow)
    float m = kNoRef;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, stats[w][r][0]);
    float y0 = 0.f, y1 = 0.f, L = 0.f;
    if (t < it.live && m != kNoRef) {
      float add = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float a = ex2_approx(stats[w][r][0] - m);
        const float2 v = *reinterpret_cast<const float2*>(&sums[w][r][C::GS * (f / (W / 8)) + f % (W / 8)]);
        L = fmaf(a, stats[w][r][1], L);
        add = fmaf(a, stats[w][r][2], add);
        y0 = fmaf(a, v.x, y0);
        y1 = fmaf(a, v.y, y1);
      }
      y0 += add;
      y1 += add;
    }
    if (!whole) {
      if (f == 0) {
        p.part_m[first_part + out] = L == 0.f ? -INFINITY : m - kLift;
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
          L == 0.f ? -INFINITY : (m - kLift + __log2f(L)) * 0.69314718055994531f;
  }
}

// Calls f with the kernel's configuration for R rows per key head of d features.
template <typename F>
void with_config(int d, int R, F&& f) {
  if (d <= 64) {
    if (R <= 8) f(Q4Cfg<64, 1, 32, 5>{});
    else f(Q4Cfg<64, 2, 32, 4>{});
  } else if (d <= 128) {
    if (R <= 8) f(Q4Cfg<128, 1, 32, 4>{});
    else f(Q4Cfg<128, 2, 32, 2>{});
  } else {
    f(Q4Cfg<256, 1, 16, 3>{});
  }
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
  const dim3 grid(static_cast<unsigned>(p.B * p.units * p.n_splits));
  with_config(p.d, p.T * p.G, [&](auto cfg) {
    e = launch_serialized(rows_q4_kernel<decltype(cfg)>, grid, dim3(32 * kWarps), 0, stream, p);
  });
  if (info) {
    info->kernels = 1;
    info->grid = static_cast<int>(grid.x);
    info->block = 32 * kWarps;
    info->smem = 0;
  }
  return e;
}

}  // namespace mha

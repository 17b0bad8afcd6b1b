// One decode step over a short 8-bit cache on the CUDA cores.
//
//   s_j = scale q . k_j 2^ek_j,   o = sum_j 2^(s_j - m) v_j 2^ev_j / sum_j 2^(s_j - m)
//
// A step of one or two query rows per key head over a few hundred keys has some 20 KB
// to read per head: what a tensor-core CTA sets up for it (barriers, tensor memory,
// pipelines between its roles) takes longer than reading it.  Here a CTA of four warps
// has a key head; a key's row is read by GS lanes, 16 codes each, so a warp's loads
// are 512 contiguous bytes per array where heads are that wide or lie side by side,
// and K, V and scales of STEP keys per lane group are in flight at once.  Every group
// of lanes keeps its own maximum, sum and sums of V in float32 registers (codes and
// scales are exact there), and the groups are merged once at the end.
//
// Work per pair of codes: one conversion to two halves, two to float32, two fused
// multiply-adds per row, so the arithmetic of 128 x 8 heads x 136 keys (mean) of 64
// features is about 1 us spread over the machine: latency (lengths, keys, merge)
// bounds it, 9.2 us from DRAM (7.4 with the cache in L2) where the tensor cores' form
// takes 17.6 and the bytes alone 2.7.
#include <cuda_bf16.h>

#include "fp8.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace mha {
namespace {

constexpr int kShortWarps = 4;
constexpr float kRoom = 16.f;  // weights are 2^-kRoom at the maximum: 2^16 keys of the largest float32 do not overflow

__device__ __forceinline__ void codes_to_float(uint32_t x, float* y) {
  const uint32_t a = e4m3x2_to_half2(static_cast<uint16_t>(x)), b = e4m3x2_to_half2(static_cast<uint16_t>(x >> 16));
  y[0] = half_lo(a);
  y[1] = half_hi(a);
  y[2] = half_lo(b);
  y[3] = half_hi(b);
}

// GS lanes per key row (16 GS >= d), NR query rows.
template <int GS, int NR>
__global__ void __launch_bounds__(32 * kShortWarps) rows_short_kernel(const __grid_constant__ RowsParams p) {
  // Keys in flight per group of lanes: more cost registers, and with them CTAs per SM
  // (from DRAM, 64 features: 128 x 8 heads x 16 to 256 keys one 9.8 us, two 9.2, four
  // 11.1; 1 x 8 heads x 256 keys 4.8, 4.6 and 4.3).
  constexpr int STEP = 2;
  constexpr int GROUPS = 32 / GS;      // keys side by side in a warp
  constexpr int KEYS = kShortWarps * GROUPS;
  __shared__ float o_s[kShortWarps][NR][GS * 16];
  __shared__ float ml_s[kShortWarps][NR][2];
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int group = lane / GS, sub = lane % GS;
  const int hk = static_cast<int>(blockIdx.x) % p.H_kv, b = static_cast<int>(blockIdx.x) / p.H_kv;
  griddep_wait();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // (with a drafted token: its key too, if it sees itself; a sequence without one
  // reads nothing)
  int prefix, live;
  int end = seq_end(p, b, &prefix, &live);
  if (p.drafts && p.tree_mask && end > prefix) end = prefix + static_cast<int>(__ldg(p.tree_mask + b) & 1);
  const bool has = 16 * sub < p.d;
  const long long q_row = static_cast<long long>(b) * p.H + hk * NR;
  float q[NR][16];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    uint4 v[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (has) {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + (q_row + r) * p.d) + 2 * sub;
      v[0] = __ldg(src);
      v[1] = __ldg(src + 1);
    }
    const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      q[r][2 * x] = bf16_lo(w[x]) * p.scale_log2;
      q[r][2 * x + 1] = bf16_hi(w[x]) * p.scale_log2;
    }
  }
  const long long key_bytes = static_cast<long long>(p.H_kv) * p.d;
  const long long first = static_cast<long long>(b) * p.Lk * key_bytes + hk * p.d + 16 * sub;
  const uint8_t* k_at = static_cast<const uint8_t*>(p.k_codes) + first;
  const uint8_t* v_at = static_cast<const uint8_t*>(p.v_codes) + first;
  const long long scales = (static_cast<long long>(b) * p.H_kv + hk) * p.Lk;

  float m[NR], l[NR], o[NR][16];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int x = 0; x < 16; ++x) o[r][x] = 0.f;
  }
  for (int key0 = warp * GROUPS; key0 < end; key0 += STEP * KEYS) {
    uint4 k4[STEP], v4[STEP];
    uint32_t kb[STEP], vb[STEP];
#pragma unroll
    for (int i = 0; i < STEP; ++i) {
      const int key = key0 + i * KEYS + group;
      k4[i] = v4[i] = make_uint4(0, 0, 0, 0);
      kb[i] = vb[i] = 127;
      if (key < end) {
        if (has) {
          k4[i] = __ldg(reinterpret_cast<const uint4*>(k_at + key * key_bytes));
          v4[i] = __ldg(reinterpret_cast<const uint4*>(v_at + key * key_bytes));
        }
        kb[i] = __ldg(p.k_scale + scales + key);
        vb[i] = __ldg(p.v_scale + scales + key);
      }
    }
    float s[NR][STEP];
#pragma unroll
    for (int i = 0; i < STEP; ++i) {
      const uint32_t w[4] = {k4[i].x, k4[i].y, k4[i].z, k4[i].w};
      float k[16];
#pragma unroll
      for (int x = 0; x < 4; ++x) codes_to_float(w[x], k + 4 * x);
      const bool valid = key0 + i * KEYS + group < end;
      const float f = __uint_as_float(kb[i] << 23);
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        float a = 0.f, c = 0.f;
#pragma unroll
        for (int x = 0; x < 16; x += 2) {
          a = fmaf(q[r][x], k[x], a);
          c = fmaf(q[r][x + 1], k[x + 1], c);
        }
        a += c;
#pragma unroll
        for (int z = 1; z < GS; z <<= 1) a += __shfl_xor_sync(0xffffffffu, a, z);
        s[r][i] = valid ? a * f : -INFINITY;
      }
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float top = m[r];
#pragma unroll
      for (int i = 0; i < STEP; ++i) top = fmaxf(top, s[r][i]);
      const float by = top == -INFINITY ? 0.f : ex2_approx(m[r] - top);  // (0 for a group's first key)
      m[r] = top;
      l[r] *= by;
#pragma unroll
      for (int x = 0; x < 16; ++x) o[r][x] *= by;
    }
#pragma unroll
    for (int i = 0; i < STEP; ++i) {
      const uint32_t w[4] = {v4[i].x, v4[i].y, v4[i].z, v4[i].w};
      float v[16];
#pragma unroll
      for (int x = 0; x < 4; ++x) codes_to_float(w[x], v + 4 * x);
      const float f = __uint_as_float(vb[i] << 23);
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float e = s[r][i] == -INFINITY ? 0.f : ex2_approx(s[r][i] - m[r] - kRoom);
        l[r] += e;
        const float a = e * f;
#pragma unroll
        for (int x = 0; x < 16; ++x) o[r][x] = fmaf(a, v[x], o[r][x]);
      }
    }
  }
  // ---- merge: the groups of a warp, then the warps
#pragma unroll
  for (int r = 0; r < NR; ++r) {
#pragma unroll
    for (int z = GS; z < 32; z <<= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m[r], z), l2 = __shfl_xor_sync(0xffffffffu, l[r], z);
      const float top = fmaxf(m[r], m2);
      const float a = m[r] == -INFINITY ? 0.f : ex2_approx(m[r] - top);
      const float c = m2 == -INFINITY ? 0.f : ex2_approx(m2 - top);
      m[r] = top;
      l[r] = fmaf(l[r], a, l2 * c);
#pragma unroll
      for (int x = 0; x < 16; ++x) o[r][x] = fmaf(o[r][x], a, __shfl_xor_sync(0xffffffffu, o[r][x], z) * c);
    }
    if (group == 0) {
#pragma unroll
      for (int x = 0; x < 16; x += 4)
        *reinterpret_cast<float4*>(&o_s[warp][r][16 * sub + x]) =
            make_float4(o[r][x], o[r][x + 1], o[r][x + 2], o[r][x + 3]);
      if (sub == 0) {
        ml_s[warp][r][0] = m[r];
        ml_s[warp][r][1] = l[r];
      }
    }
  }
  __syncthreads();
  for (int x = static_cast<int>(threadIdx.x) * 2; x < NR * p.d; x += 2 * 32 * kShortWarps) {
    const int r = x / p.d, f = x - r * p.d;
    float top = -INFINITY, L = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll
    for (int w = 0; w < kShortWarps; ++w) top = fmaxf(top, ml_s[w][r][0]);
#pragma unroll
    for (int w = 0; w < kShortWarps; ++w) {
      const float a = ml_s[w][r][0] == -INFINITY ? 0.f : ex2_approx(ml_s[w][r][0] - top);
      L = fmaf(a, ml_s[w][r][1], L);
      y0 = fmaf(a, o_s[w][r][f], y0);
      y1 = fmaf(a, o_s[w][r][f + 1], y1);
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + (q_row + r) * p.d + f) =
        pack_bf16x2(y0 * inv, y1 * inv);
    if (p.lse && f == 0)
      p.lse[q_row + r] = L > 0.f ? (top + kRoom + __log2f(L)) * 0.69314718055994531f : -INFINITY;
  }
}

template <int GS>
cudaError_t launch_short(const RowsParams& p, cudaStream_t stream, LaunchInfo* info) {
  const dim3 grid(static_cast<unsigned>(p.B * p.units));
  const cudaError_t e = launch_serialized(p.G == 1 ? rows_short_kernel<GS, 1> : rows_short_kernel<GS, 2>, grid,
                                          dim3(32 * kShortWarps), 0, stream, p);
  if (info) {
    info->kernels = 1;
    info->grid = static_cast<int>(grid.x);
    info->block = 32 * kShortWarps;
    info->smem = 0;
  }
  return e;
}

}  // namespace

cudaError_t launch_rows_short(const RowsParams& p, cudaStream_t stream, LaunchInfo* info) {
  return p.d <= 64 ? launch_short<4>(p, stream, info)
                   : (p.d <= 128 ? launch_short<8>(p, stream, info) : launch_short<16>(p, stream, info));
}

}  // namespace mha

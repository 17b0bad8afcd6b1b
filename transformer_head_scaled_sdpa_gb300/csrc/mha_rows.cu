// mha_rows.cu -- attention of a few query rows per sequence over a key/value
// cache: the decode step over the 8-bit cache and the step of a tree of
// drafted tokens over either cache, sm_103a.
#include <cuda_bf16.h>

#include "fp8.cuh"
#include "kernels.h"

namespace mha {
namespace {

// One warp per (sequence, drafted token, head).
template <bool F8>
__global__ void __launch_bounds__(256) rows_simple_kernel(const __grid_constant__ RowsParams p) {
  griddep_wait();
  const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= static_cast<long long>(p.B) * p.T * p.H) return;
  const int h = static_cast<int>(row % p.H);
  const int t = static_cast<int>(row / p.H % p.T);
  const int b = static_cast<int>(row / p.H / p.T);
  const int hk = h / p.G;
  int n = __ldg(p.prefix_lens + b);
  n = n < 0 ? 0 : (n > p.Lk ? p.Lk : n);
  int live = p.T;
  if (p.draft_lens) {
    live = __ldg(p.draft_lens + b);
    live = live < 0 ? 0 : (live > p.T ? p.T : live);
  }
  const int end = t < live ? min(p.Lk, n + (p.drafts ? live : 0)) : 0;
  float q[8], acc[8] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = lane + 32 * i;
    q[i] = e < p.d ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[row * p.d + e]) * p.scale_log2 : 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < end; ++j) {
    if (j >= n) {
      const int x = j - n;
      const bool sees = p.tree_mask ? (p.tree_mask[(static_cast<long long>(b) * p.T + t) * p.words + x / 64] >> (x % 64)) & 1
                                    : x <= t;
      if (!sees) continue;
    }
    const long long kr = ((static_cast<long long>(b) * p.Lk + j) * p.H_kv + hk) * p.d;
    float kf = 1.f, vf = 1.f;
    if (F8) {
      const long long sr = (static_cast<long long>(b) * p.H_kv + hk) * p.Lk + j;
      kf = pow2i(p.k_scale[sr] - 127);
      vf = pow2i(p.v_scale[sr] - 127);
    }
    auto at = [&](const void* c, long long i) {
      if (F8) return half_lo(e4m3x2_to_half2(static_cast<const uint8_t*>(c)[i]));
      return __bfloat162float(static_cast<const __nv_bfloat16*>(c)[i]);
    };
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane + 32 * i < p.d) s = fmaf(q[i], at(p.k, kr + lane + 32 * i), s);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= kf;
    const float mn = fmaxf(m, s), a = exp2f(m - mn), w = exp2f(s - mn);
    l = l * a + w;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane + 32 * i < p.d) acc[i] = acc[i] * a + w * vf * at(p.v, kr + lane + 32 * i);
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (lane + 32 * i < p.d)
      static_cast<__nv_bfloat16*>(p.out)[row * p.d + lane + 32 * i] = __float2bfloat16_rn(acc[i] * inv);
  if (p.lse && lane == 0)
    p.lse[(static_cast<long long>(b) * p.H + h) * p.T + t] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

int rows_splits(int, int, int, int, int, int, bool) { return 1; }

int rows_kernel_width(int d, bool f8) {
  if (f8) return d <= 128 ? 128 : 256;
  return d <= 64 ? 64 : (d <= 128 ? 128 : 256);
}

cudaError_t launch_rows(const RowsParams& p, cudaStream_t stream, LaunchInfo* info) {
  const long long rows = static_cast<long long>(p.B) * p.T * p.H;
  const dim3 grid(static_cast<unsigned>((rows + 7) / 8));
  const cudaError_t e = p.k_scale ? launch_serialized(rows_simple_kernel<true>, grid, dim3(256), 0, stream, p)
                                  : launch_serialized(rows_simple_kernel<false>, grid, dim3(256), 0, stream, p);
  if (info) {
    info->kernels = 1;
    info->grid = static_cast<int>(grid.x);
    info->block = 256;
  }
  return e;
}

}  // namespace mha

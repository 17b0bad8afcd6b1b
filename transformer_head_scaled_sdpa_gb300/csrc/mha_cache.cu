// mha_cache.cu -- the 8-bit key/value cache: rows quantised as they are
// written, and read back, sm_103a.
//
// A decoder that emits one token per step keeps the keys and values of the
// steps before (cookipedia article, section "Transformer 全体"; D2L notes, the
// three kinds of attention, decoder layer A).  Here they are kept in 8 bits:
// per position and head one row of d e4m3 codes and one byte, the row's
// power-of-two scale (fp8.cuh):
//     write  e = min { e >= -64 : max |x| <= 448 * 2^e },  c = rn_e4m3(x * 2^-e)
//     read   x' = c * 2^e   (exact in bf16)
// Codes are [B, Lk, H, d] like the bf16 caches; scales are [B, H, Lk], so a
// reader that streams one head's positions streams its scales too.
//
// Both are bound by memory: 2 * 2d bytes on the bf16 side and 2 * (d + 1) on
// the cache's per position and head.  One block takes a tile of positions x
// heads of one sequence; a row is handled by a group of 1 to 16 lanes, sixteen
// elements (two 16-byte pieces of bf16) to a lane, and a lane keeps the K and V
// pieces of two positions in flight.  Rows are addressed by adding strides: with
// a division per row, and eight elements to a lane, issuing instructions bounded
// both (4 x 1024-2048 positions x 96 heads x 128 features: 120 us written, 92 us
// read, against 70 and 70: 0.96 of the copy rate).
#include <cuda_bf16.h>

#include "fp8.cuh"
#include "kernels.h"

namespace mha {
namespace {

constexpr int kThreads = 256;
constexpr int kTileTokens = 32;  // positions per block: one 32-byte sector of a head's scales
constexpr int kTileHeads = 8;    // heads per block

// What a thread works on: pieces `sub` and `sub + GS` (16 bytes of bf16 each) of
// the rows of head `h` at the tile's positions t0 + t, t0 + t + step, ...
struct Rows {
  int b, h, t0, t, nt, step;
  bool head_ok;
};

template <int GS>
__device__ __forceinline__ Rows thread_rows(const CacheParams& p) {
  const unsigned head_tiles = (p.H + kTileHeads - 1) / kTileHeads;
  const unsigned token_tiles = (p.T + kTileTokens - 1) / kTileTokens;
  const unsigned x = blockIdx.x / head_tiles;
  const int group = static_cast<int>(threadIdx.x) / GS;
  Rows r;
  r.b = static_cast<int>(x / token_tiles);
  r.t0 = static_cast<int>(x % token_tiles) * kTileTokens;
  r.h = static_cast<int>(blockIdx.x % head_tiles) * kTileHeads + group % kTileHeads;
  r.head_ok = r.h < p.H;
  r.t = group / kTileHeads;
  r.nt = min(kTileTokens, p.T - r.t0);
  r.step = static_cast<int>(blockDim.x) / (GS * kTileHeads);
  return r;
}

// max |x| of eight bf16 (NaN passed over: it stays a NaN code of its own)
__device__ __forceinline__ __nv_bfloat162 abs_max8(const uint4& x) {
  const __nv_bfloat162* v = reinterpret_cast<const __nv_bfloat162*>(&x);
  return __hmax2(__hmax2(__habs2(v[0]), __habs2(v[1])), __hmax2(__habs2(v[2]), __habs2(v[3])));
}

// Four bf16 (two words) times `f` to e4m3 codes.
__device__ __forceinline__ uint32_t codes4(uint32_t a, uint32_t b, float f) {
  float x0, x1, x2, x3;
  mul2(x0, x1, bf16_lo(a), bf16_hi(a), f, f);
  mul2(x2, x3, bf16_lo(b), bf16_hi(b), f, f);
  return pack_e4m3x2(x0, x1) | (static_cast<uint32_t>(pack_e4m3x2(x2, x3)) << 16);
}

// GS: lanes per row, the power of two >= d / 16
template <int GS>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const __grid_constant__ CacheParams p) {
  griddep_wait();
  const Rows r = thread_rows<GS>(p);
  const int sub = static_cast<int>(threadIdx.x) % GS;
  const bool has0 = 8 * sub < p.d, has1 = 8 * (sub + GS) < p.d;
  const int start = __ldg(p.lens + r.b);
  int count = p.T;
  if (p.counts) {
    const int c = __ldg(p.counts + r.b);
    count = c < 0 ? 0 : (c < p.T ? c : p.T);
  }
  // positions first .. last - 1 of the tile are written
  const long long at0 = static_cast<long long>(start) + r.t0;
  const int first = at0 < 0 ? static_cast<int>(min(-at0, static_cast<long long>(r.nt))) : 0;
  const int last = static_cast<int>(
      max(0ll, min(static_cast<long long>(min(r.nt, count - r.t0)), static_cast<long long>(p.Lk) - at0)));
  const long long src_row = p.seq_elems * r.b + static_cast<long long>(r.h) * p.d + 8 * sub;
  const uint16_t* src[2] = {static_cast<const uint16_t*>(p.k) + src_row,
                            static_cast<const uint16_t*>(p.v) + src_row};
  const long long dst_row =
      ((static_cast<long long>(r.b) * p.Lk + at0) * p.H + r.h) * p.d + 8 * sub;
  uint8_t* dst[2] = {static_cast<uint8_t*>(p.k_cache) + dst_row, static_cast<uint8_t*>(p.v_cache) + dst_row};
  const long long scale_row = (static_cast<long long>(r.b) * p.H + r.h) * p.Lk + at0;
  const long long pos_bytes = static_cast<long long>(p.H) * p.d;  // bytes between positions of the cache
  // (the loop's bound is the same for every lane: the shuffles are the whole
  // warp's)
  for (int base = 0; base < r.nt; base += 2 * r.step) {
    uint4 x[2][2][2] = {};  // [position][K, V][piece]
    bool on[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = base + u * r.step + r.t;
      on[u] = r.head_ok && t >= first && t < last;
      if (!on[u]) continue;
      const long long o = p.row_elems * (r.t0 + t);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (has0) x[u][c][0] = __ldg(reinterpret_cast<const uint4*>(src[c] + o));
        if (has1) x[u][c][1] = __ldg(reinterpret_cast<const uint4*>(src[c] + o + 8 * GS));
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = base + u * r.step + r.t;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const __nv_bfloat162 m2 = __hmax2(abs_max8(x[u][c][0]), abs_max8(x[u][c][1]));
        float amax = fmaxf(fmaxf(__low2float(m2), __high2float(m2)), 0.f);  // (0: all NaN)
#pragma unroll
        for (int o = 1; o < GS; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (!on[u]) continue;
        const int s = row_scale_byte(amax);
        const float f = pow2i(127 - s);
        uint8_t* to = dst[c] + t * pos_bytes;
        const uint4 a = x[u][c][0], b = x[u][c][1];
        if (has0) *reinterpret_cast<uint2*>(to) = make_uint2(codes4(a.x, a.y, f), codes4(a.z, a.w, f));
        if (has1) *reinterpret_cast<uint2*>(to + 8 * GS) = make_uint2(codes4(b.x, b.y, f), codes4(b.z, b.w, f));
        if (sub == 0) (c == 0 ? p.k_scale : p.v_scale)[scale_row + t] = static_cast<uint8_t>(s);
      }
    }
  }
}

// Four codes times `f` to bf16 (two words).
__device__ __forceinline__ uint2 values4(uint32_t c, float f) {
  const uint32_t a = e4m3x2_to_half2(static_cast<uint16_t>(c)), b = e4m3x2_to_half2(static_cast<uint16_t>(c >> 16));
  float x0, x1, x2, x3;
  mul2(x0, x1, half_lo(a), half_hi(a), f, f);
  mul2(x2, x3, half_lo(b), half_hi(b), f, f);
  return make_uint2(pack_bf16x2(x0, x1), pack_bf16x2(x2, x3));
}

template <int GS>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ CacheParams p) {
  griddep_wait();
  const Rows r = thread_rows<GS>(p);
  const int sub = static_cast<int>(threadIdx.x) % GS;
  const bool has0 = 8 * sub < p.d, has1 = 8 * (sub + GS) < p.d;
  if (!r.head_ok || !has0) return;
  const int last = min(r.nt, max(__ldg(p.lens + r.b), 0) - r.t0);
  const long long row = ((static_cast<long long>(r.b) * p.Lk + r.t0) * p.H + r.h) * p.d + 8 * sub;
  const uint8_t* src[2] = {static_cast<const uint8_t*>(p.k_cache) + row,
                           static_cast<const uint8_t*>(p.v_cache) + row};
  uint16_t* dst[2] = {static_cast<uint16_t*>(p.k_out) + row, static_cast<uint16_t*>(p.v_out) + row};
  const long long scale_row = (static_cast<long long>(r.b) * p.H + r.h) * p.Lk + r.t0;
  const uint8_t* scale[2] = {p.k_scale + scale_row, p.v_scale + scale_row};
  const long long pos = static_cast<long long>(p.H) * p.d;  // elements between positions
  for (int t0 = r.t; t0 < last; t0 += 2 * r.step) {
    uint2 x[2][2][2];
    uint32_t s[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = t0 + u * r.step;
      if (t >= last) continue;
      const long long o = t * pos;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        x[u][c][0] = __ldg(reinterpret_cast<const uint2*>(src[c] + o));
        if (has1) x[u][c][1] = __ldg(reinterpret_cast<const uint2*>(src[c] + o + 8 * GS));
        s[u][c] = __ldg(scale[c] + t);
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = t0 + u * r.step;
      if (t >= last) continue;
      const long long o = t * pos;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        // a scale of 2^-127 (byte 0) is no float32 power of two: such a row
        // reads as 0 (written rows have bytes 63 to 247)
        const float f = __uint_as_float(s[u][c] << 23);
        uint2 a = values4(x[u][c][0].x, f), b = values4(x[u][c][0].y, f);
        *reinterpret_cast<uint4*>(dst[c] + o) = make_uint4(a.x, a.y, b.x, b.y);
        if (has1) {
          a = values4(x[u][c][1].x, f);
          b = values4(x[u][c][1].y, f);
          *reinterpret_cast<uint4*>(dst[c] + o + 8 * GS) = make_uint4(a.x, a.y, b.x, b.y);
        }
      }
    }
  }
}

template <int GS>
cudaError_t launch_gs(const CacheParams& p, bool write, unsigned blocks, cudaStream_t s, LaunchInfo* info) {
  // as many positions at a time as the block has threads for, or as there are
  const int fit = kThreads / (GS * kTileHeads);
  int threads = (p.T < fit ? p.T : fit) * GS * kTileHeads;
  threads = (threads + 31) / 32 * 32;
  if (info) {
    info->kernels = 1;
    info->grid = static_cast<int>(blocks);
    info->block = threads;
    info->smem = 0;
  }
  return write ? launch_serialized(cache_write_kernel<GS>, dim3(blocks), dim3(threads), 0, s, p)
               : launch_serialized(cache_read_kernel<GS>, dim3(blocks), dim3(threads), 0, s, p);
}

}  // namespace

long long cache_blocks(int B, int T, int H) {
  return static_cast<long long>(B) * ((T + kTileTokens - 1) / kTileTokens) *
         ((H + kTileHeads - 1) / kTileHeads);
}

cudaError_t launch_cache(const CacheParams& p, bool write, cudaStream_t stream, LaunchInfo* info) {
  const unsigned blocks = static_cast<unsigned>(cache_blocks(p.B, p.T, p.H));
  const int lanes = p.d / 16;
  if (lanes <= 1) return launch_gs<1>(p, write, blocks, stream, info);
  if (lanes <= 2) return launch_gs<2>(p, write, blocks, stream, info);
  if (lanes <= 4) return launch_gs<4>(p, write, blocks, stream, info);
  if (lanes <= 8) return launch_gs<8>(p, write, blocks, stream, info);
  return launch_gs<16>(p, write, blocks, stream, info);
}

}  // namespace mha

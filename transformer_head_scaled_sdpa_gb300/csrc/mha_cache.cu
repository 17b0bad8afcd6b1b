// mha_cache.cu -- the 8-bit and the 4-bit key/value cache: rows quantised as
// they are written, and read back, sm_103a.
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
//
// In 4 bits (q4.cuh: the format and how its codes are decided) a row is d / 2 bytes and two
// bf16 numbers; the tiles, lanes and strides are the same, with sixteen positions to a tile
// (78 us with 32, 77 with 8, against 73 for the second sizes below).  A read is bound
// by memory, a write by instructions (0.71 of the issue slots: per element a comparison for
// the smallest and the largest, a product, and its place among the codes): 64 x 512 x 8
// heads of 64 features, half of them full, written and read in 32 us (126 MB, 3.9 TB/s); 4 x
// 300 to 512 tokens x 96 heads of 128 written and 2,085 read back in 74 (5.3 TB/s).
#include <cuda_bf16.h>

#include "fp8.cuh"
#include "kernels.h"
#include "q4.cuh"

namespace mha {
namespace {

constexpr int kThreads = 256;
constexpr int kTileTokens = 32;  // positions per block: one 32-byte sector of a head's scales
constexpr int kTileTokensQ4 = 16;  // 4 bits: at most
constexpr int kTileHeads = 8;    // heads per block

// What a thread works on: pieces `sub` and `sub + GS` (16 bytes of bf16 each) of
// the rows of head `h` at the tile's positions t0 + t, t0 + t + step, ...
struct Rows {
  int b, h, t0, t, nt, step;
  bool head_ok;
};

template <int GS, int TOKENS = kTileTokens>
__device__ __forceinline__ Rows thread_rows(const CacheParams& p) {
  const unsigned head_tiles = (p.H + kTileHeads - 1) / kTileHeads;
  const unsigned token_tiles = (p.T + TOKENS - 1) / TOKENS;
  const unsigned x = blockIdx.x / head_tiles;
  const int group = static_cast<int>(threadIdx.x) / GS;
  Rows r;
  r.b = static_cast<int>(x / token_tiles);
  r.t0 = static_cast<int>(x % token_tiles) * TOKENS;
  r.h = static_cast<int>(blockIdx.x % head_tiles) * kTileHeads + group % kTileHeads;
  r.head_ok = r.h < p.H;
  r.t = group / kTileHeads;
  r.nt = min(TOKENS, p.T - r.t0);
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
        if (sub == 0) static_cast<uint8_t*>(c == 0 ? p.k_scale : p.v_scale)[scale_row + t] = static_cast<uint8_t>(s);
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
  const uint8_t* scale[2] = {static_cast<const uint8_t*>(p.k_scale) + scale_row,
                             static_cast<const uint8_t*>(p.v_scale) + scale_row};
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

// ---------------------------------------------------------------------------
// 4 bits (q4.cuh): the same tiles of positions x heads, eight codes to a word.
// ---------------------------------------------------------------------------

// (min, -max) of eight bf16 (a NaN stays).
__device__ __forceinline__ __nv_bfloat162 low_high8(const uint4& x) {
  const __nv_bfloat162* v = reinterpret_cast<const __nv_bfloat162*>(&x);
  const __nv_bfloat162 lo = __hmin2_nan(__hmin2_nan(v[0], v[1]), __hmin2_nan(v[2], v[3]));
  const __nv_bfloat162 hi = __hmax2_nan(__hmax2_nan(v[0], v[1]), __hmax2_nan(v[2], v[3]));
  return __halves2bfloat162(__hmin_nan(__low2bfloat16(lo), __high2bfloat16(lo)),
                            __hneg(__hmax_nan(__low2bfloat16(hi), __high2bfloat16(hi))));
}

// Eight bf16 to a word of codes.
__device__ __forceinline__ uint32_t codes8(const uint4& x, const RowQ4& r) {
  const float y[8] = {bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y),
                      bf16_lo(x.z), bf16_hi(x.z), bf16_lo(x.w), bf16_hi(x.w)};
  return codes_q4(y, r);
}

// GS: lanes per row, the power of two >= d / 16
template <int GS, int TOKENS>
__global__ void __launch_bounds__(kThreads, 4) cache_write_q4_kernel(const __grid_constant__ CacheParams p) {
  griddep_wait();
  const Rows r = thread_rows<GS, TOKENS>(p);
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
  const long long pos_bytes = static_cast<long long>(p.H) * (p.d / 2);  // between positions of the cache
  const long long dst_row = (static_cast<long long>(r.b) * p.Lk + at0) * pos_bytes +
                            static_cast<long long>(r.h) * (p.d / 2) + 4 * sub;
  uint8_t* dst[2] = {static_cast<uint8_t*>(p.k_cache) + dst_row, static_cast<uint8_t*>(p.v_cache) + dst_row};
  const long long scale_row = (static_cast<long long>(r.b) * p.H + r.h) * p.Lk + at0;
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
        // (a lane without a piece has +-infinity, which loses to every value)
        __nv_bfloat162 m = __halves2bfloat162(__ushort_as_bfloat16(0x7f80), __ushort_as_bfloat16(0x7f80));
        if (has0) m = low_high8(x[u][c][0]);
        if (has1) m = __hmin2_nan(m, low_high8(x[u][c][1]));
#pragma unroll
        for (int o = 1; o < GS; o <<= 1) m = __hmin2_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (!on[u]) continue;
        const RowQ4 row = row_q4(__low2float(m), -__high2float(m));
        const bool bad = row.lo != row.lo;
        uint8_t* to = dst[c] + t * pos_bytes;
        if (has0) *reinterpret_cast<uint32_t*>(to) = bad ? 0 : codes8(x[u][c][0], row);
        if (has1) *reinterpret_cast<uint32_t*>(to + 4 * GS) = bad ? 0 : codes8(x[u][c][1], row);
        if (sub == 0)
          static_cast<uint32_t*>(c == 0 ? p.k_scale : p.v_scale)[scale_row + t] =
              (__float_as_uint(row.lo) >> 16) | (__float_as_uint(row.step) & 0xffff0000u);
      }
    }
  }
}

// Eight codes to bf16: lo + c * step, rounded to float32 and then to bf16.
__device__ __forceinline__ uint4 values8(uint32_t c, float lo, float step) {
  uint32_t y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // (128 + c as a bf16 number has the code in its last bits)
    const float a = __uint_as_float(0x43000000u | (((c >> (8 * i)) & 15u) << 16));
    const float b = __uint_as_float(0x43000000u | (((c >> (8 * i + 4)) & 15u) << 16));
    float x0, x1;
    add2(x0, x1, a, b, -128.f, -128.f);
    fma2(x0, x1, x0, x1, step, step, lo, lo);
    y[i] = pack_bf16x2(x0, x1);
  }
  return make_uint4(y[0], y[1], y[2], y[3]);
}

template <int GS, int TOKENS>
__global__ void __launch_bounds__(kThreads) cache_read_q4_kernel(const __grid_constant__ CacheParams p) {
  griddep_wait();
  const Rows r = thread_rows<GS, TOKENS>(p);
  const int sub = static_cast<int>(threadIdx.x) % GS;
  const bool has0 = 8 * sub < p.d, has1 = 8 * (sub + GS) < p.d;
  if (!r.head_ok || !has0) return;
  const int last = min(r.nt, max(__ldg(p.lens + r.b), 0) - r.t0);
  const long long row = ((static_cast<long long>(r.b) * p.Lk + r.t0) * p.H + r.h) * p.d + 8 * sub;
  const uint8_t* src[2] = {static_cast<const uint8_t*>(p.k_cache) + row / 2,
                           static_cast<const uint8_t*>(p.v_cache) + row / 2};
  uint16_t* dst[2] = {static_cast<uint16_t*>(p.k_out) + row, static_cast<uint16_t*>(p.v_out) + row};
  const long long scale_row = (static_cast<long long>(r.b) * p.H + r.h) * p.Lk + r.t0;
  const uint32_t* scale[2] = {static_cast<const uint32_t*>(p.k_scale) + scale_row,
                              static_cast<const uint32_t*>(p.v_scale) + scale_row};
  const long long pos = static_cast<long long>(p.H) * p.d;  // elements between positions
  for (int t0 = r.t; t0 < last; t0 += 2 * r.step) {
    uint32_t x[2][2][2], s[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = t0 + u * r.step;
      if (t >= last) continue;
      const long long o = t * pos / 2;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        x[u][c][0] = __ldg(reinterpret_cast<const uint32_t*>(src[c] + o));
        if (has1) x[u][c][1] = __ldg(reinterpret_cast<const uint32_t*>(src[c] + o + 4 * GS));
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
        const float lo = bf16_lo(s[u][c]), step = bf16_hi(s[u][c]);
        *reinterpret_cast<uint4*>(dst[c] + o) = values8(x[u][c][0], lo, step);
        if (has1) *reinterpret_cast<uint4*>(dst[c] + o + 8 * GS) = values8(x[u][c][1], lo, step);
      }
    }
  }
}

template <int GS>
cudaError_t launch_gs(const CacheParams& p, CacheKind kind, bool write, int tile, unsigned blocks, cudaStream_t s,
                      LaunchInfo* info) {
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
  auto* kernel = write ? cache_write_kernel<GS> : cache_read_kernel<GS>;
  if (kind == kCacheQ4) {
    if (tile == 4) kernel = write ? cache_write_q4_kernel<GS, 4> : cache_read_q4_kernel<GS, 4>;
    else if (tile == 8) kernel = write ? cache_write_q4_kernel<GS, 8> : cache_read_q4_kernel<GS, 8>;
    else kernel = write ? cache_write_q4_kernel<GS, 16> : cache_read_q4_kernel<GS, 16>;
  }
  return launch_serialized(kernel, dim3(blocks), dim3(threads), 0, s, p);
}

}  // namespace

static long long blocks_of(int B, int T, int H, int tokens) {
  return static_cast<long long>(B) * ((T + tokens - 1) / tokens) * ((H + kTileHeads - 1) / kTileHeads);
}

long long cache_blocks(CacheKind kind, int B, int T, int H) {
  return blocks_of(B, T, H, kind == kCacheQ4 ? kTileTokensQ4 : kTileTokens);
}

cudaError_t launch_cache(const CacheParams& p, CacheKind kind, bool write, cudaStream_t stream, LaunchInfo* info) {
  int tile = kind == kCacheQ4 ? kTileTokensQ4 : kTileTokens;
  // Few rows in 4 bits: tiles of 8 or 4 positions as long as that makes no more than four blocks
  // to an SM.  us with 16, 8 and 4, written: 4 x 16 tokens x 96 heads of 128 features 6.6 4.7
  // 4.2, 2,000 x 2 of 256 10.7 7.0 5.7, 2,000 x 32 of 64 (500, 1,000 and 2,000 blocks) 8.1 8.7
  // 12.5, 64 x 512 x 8 of 64 20.5 26.2 39.3; read: 2,000
  // x 2 of 256 4.8 with 16, 3.6 with 4.
  if (kind == kCacheQ4)
    while (tile > 4 && blocks_of(p.B, p.T, p.H, tile / 2) <= 4 * 152) tile /= 2;
  const unsigned blocks = static_cast<unsigned>(blocks_of(p.B, p.T, p.H, tile));
  const int lanes = p.d / 16;
  if (lanes <= 1) return launch_gs<1>(p, kind, write, tile, blocks, stream, info);
  if (lanes <= 2) return launch_gs<2>(p, kind, write, tile, blocks, stream, info);
  if (lanes <= 4) return launch_gs<4>(p, kind, write, tile, blocks, stream, info);
  if (lanes <= 8) return launch_gs<8>(p, kind, write, tile, blocks, stream, info);
  return launch_gs<16>(p, kind, write, tile, blocks, stream, info);
}

}  // namespace mha

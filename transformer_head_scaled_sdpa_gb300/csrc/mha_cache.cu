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
// heads of one sequence; a row is handled by d / 8 lanes (16 bytes of bf16, 8
// of codes each) of a group of 1 to 32, and a thread keeps kRowsInFlight rows
// in flight.
#include "fp8.cuh"
#include "kernels.h"

namespace mha {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsInFlight = 4;
constexpr int kTileTokens = 32;  // positions per block: one 32-byte sector of a head's scales
constexpr int kTileHeads = 8;    // heads per block

// What a block works on: rows r of its tile, in the order K then V, then
// position, then head (the fastest).
struct Tile {
  int b, t0, h0, nt, nh;
  int rows;  // nt * nh rows of K, as many of V
};

__device__ __forceinline__ Tile block_tile(const CacheParams& p) {
  const int head_tiles = (p.H + kTileHeads - 1) / kTileHeads;
  const int token_tiles = (p.T + kTileTokens - 1) / kTileTokens;
  unsigned x = blockIdx.x;
  Tile t;
  t.h0 = static_cast<int>(x % head_tiles) * kTileHeads;
  x /= head_tiles;
  t.t0 = static_cast<int>(x % token_tiles) * kTileTokens;
  t.b = static_cast<int>(x / token_tiles);
  t.nt = min(kTileTokens, p.T - t.t0);
  t.nh = min(kTileHeads, p.H - t.h0);
  t.rows = t.nt * t.nh;
  return t;
}

// GS: lanes per row, the power of two >= d / 8
template <int GS>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const __grid_constant__ CacheParams p) {
  griddep_wait();
  const Tile tile = block_tile(p);
  const int sub = static_cast<int>(threadIdx.x) % GS;
  const int group = static_cast<int>(threadIdx.x) / GS;
  constexpr int kGroups = kThreads / GS;
  const bool active = sub * 8 < p.d;
  const int start = __ldg(p.lens + tile.b);
  int count = p.T;
  if (p.counts) {
    const int c = __ldg(p.counts + tile.b);
    count = c < 0 ? 0 : (c < p.T ? c : p.T);
  }
  // (the loop's bound is the same for every lane: the shuffles below are the
  // whole warp's)
  for (int base = 0; base < 2 * tile.rows; base += kRowsInFlight * kGroups) {
    const int r0 = base + group;
    uint4 x[kRowsInFlight];
    long long pos[kRowsInFlight];  // -1: nothing to write
    int head[kRowsInFlight];
#pragma unroll
    for (int u = 0; u < kRowsInFlight; ++u) {
      const int r = r0 + u * kGroups;
      pos[u] = -1;
      x[u] = make_uint4(0, 0, 0, 0);
      if (r >= 2 * tile.rows) continue;
      const int rr = r < tile.rows ? r : r - tile.rows;
      const int t = tile.t0 + rr / tile.nh;
      head[u] = tile.h0 + rr % tile.nh;
      const long long at = static_cast<long long>(start) + t;
      if (t >= count || at < 0 || at >= p.Lk) continue;
      pos[u] = at;
      const uint16_t* src = static_cast<const uint16_t*>(r < tile.rows ? p.k : p.v);
      if (active)
        x[u] = __ldg(reinterpret_cast<const uint4*>(src + p.seq_elems * tile.b + p.row_elems * t +
                                                    static_cast<long long>(head[u]) * p.d + sub * 8));
    }
#pragma unroll
    for (int u = 0; u < kRowsInFlight; ++u) {
      const int r = r0 + u * kGroups;
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      float amax = 0.f;  // (fmaxf passes over NaN: it stays a NaN code of its own)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
#pragma unroll
      for (int o = 1; o < GS; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (pos[u] < 0) continue;
      const int s = row_scale_byte(amax);
      const float inv = pow2i(127 - s);
      uint32_t c[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        c[i] = pack_e4m3x2(bf16_lo(w[2 * i]) * inv, bf16_hi(w[2 * i]) * inv) |
               (static_cast<uint32_t>(pack_e4m3x2(bf16_lo(w[2 * i + 1]) * inv,
                                                  bf16_hi(w[2 * i + 1]) * inv))
                << 16);
      const bool is_k = r < tile.rows;
      uint8_t* codes = static_cast<uint8_t*>(is_k ? p.k_cache : p.v_cache);
      uint8_t* scales = is_k ? p.k_scale : p.v_scale;
      if (active)
        *reinterpret_cast<uint2*>(codes + ((static_cast<long long>(tile.b) * p.Lk + pos[u]) * p.H + head[u]) * p.d +
                                  sub * 8) = make_uint2(c[0], c[1]);
      if (sub == 0)
        scales[(static_cast<long long>(tile.b) * p.H + head[u]) * p.Lk + pos[u]] = static_cast<uint8_t>(s);
    }
  }
}

template <int GS>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ CacheParams p) {
  griddep_wait();
  const Tile tile = block_tile(p);
  const int sub = static_cast<int>(threadIdx.x) % GS;
  const int group = static_cast<int>(threadIdx.x) / GS;
  constexpr int kGroups = kThreads / GS;
  if (sub * 8 >= p.d) return;  // (no lane of another row depends on this one)
  const int count = __ldg(p.lens + tile.b);
  for (int r0 = group; r0 < 2 * tile.rows; r0 += kRowsInFlight * kGroups) {
    uint2 c[kRowsInFlight];
    int s[kRowsInFlight];
    long long row[kRowsInFlight];  // (b, position, head); -1: nothing to read
#pragma unroll
    for (int u = 0; u < kRowsInFlight; ++u) {
      const int r = r0 + u * kGroups;
      row[u] = -1;
      if (r >= 2 * tile.rows) continue;
      const int rr = r < tile.rows ? r : r - tile.rows;
      const int t = tile.t0 + rr / tile.nh, head = tile.h0 + rr % tile.nh;
      if (t >= count) continue;
      row[u] = (static_cast<long long>(tile.b) * p.Lk + t) * p.H + head;
      const bool is_k = r < tile.rows;
      c[u] = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(is_k ? p.k_cache : p.v_cache) +
                                                  row[u] * p.d + sub * 8));
      s[u] = __ldg((is_k ? p.k_scale : p.v_scale) + (static_cast<long long>(tile.b) * p.H + head) * p.Lk + t);
    }
#pragma unroll
    for (int u = 0; u < kRowsInFlight; ++u) {
      if (row[u] < 0) continue;
      // a scale of 2^-127 (byte 0) is no float32 power of two: such a row
      // reads as 0 (written rows have bytes 63 to 247)
      const float f = s[u] == 0 ? 0.f : pow2i(s[u] - 127);
      const uint32_t in[2] = {c[u].x, c[u].y};
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t h2 = e4m3x2_to_half2(static_cast<uint16_t>(in[i >> 1] >> (16 * (i & 1))));
        w[i] = pack_bf16x2(half_lo(h2) * f, half_hi(h2) * f);
      }
      void* dst = r0 + u * kGroups < tile.rows ? p.k_out : p.v_out;
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + row[u] * p.d + sub * 8) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

template <int GS>
cudaError_t launch_gs(const CacheParams& p, bool write, unsigned blocks, cudaStream_t s) {
  return write ? launch_serialized(cache_write_kernel<GS>, dim3(blocks), dim3(kThreads), 0, s, p)
               : launch_serialized(cache_read_kernel<GS>, dim3(blocks), dim3(kThreads), 0, s, p);
}

}  // namespace

long long cache_blocks(int B, int T, int H) {
  return static_cast<long long>(B) * ((T + kTileTokens - 1) / kTileTokens) *
         ((H + kTileHeads - 1) / kTileHeads);
}

cudaError_t launch_cache(const CacheParams& p, bool write, cudaStream_t stream, LaunchInfo* info) {
  const unsigned blocks = static_cast<unsigned>(cache_blocks(p.B, p.T, p.H));
  const int lanes = p.d / 8;
  cudaError_t e;
  if (lanes <= 2) e = launch_gs<2>(p, write, blocks, stream);
  else if (lanes <= 4) e = launch_gs<4>(p, write, blocks, stream);
  else if (lanes <= 8) e = launch_gs<8>(p, write, blocks, stream);
  else if (lanes <= 16) e = launch_gs<16>(p, write, blocks, stream);
  else e = launch_gs<32>(p, write, blocks, stream);
  if (info) {
    info->kernels = 1;
    info->grid = static_cast<int>(blocks);
    info->block = kThreads;
    info->smem = 0;
  }
  return e;
}

}  // namespace mha

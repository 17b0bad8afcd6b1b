// Attention of many query rows per key head over a bf16 cache, keys split over CTAs.
//
// The steps of mha_rows.cu put the keys along the tensor core's M and a unit's rows
// along its N, which suits a few rows: a tile of K is an operand as TMA wrote it,
// whatever the number of rows.  From 64 rows on that costs more than it saves: P
// goes through shared memory, K and V are read there once per block of 64 rows, and
// shared memory's 128 bytes per cycle bound the step.  Here a unit has up to 256
// rows, two tiles of 128 along M that share every tile of K and V:
//   S_g[128 x 128 keys] = Q_g K^T   (Q, K in shared memory, K-major)
//   O_g[128 x d] += P_g V           (P in tensor memory, V as loaded, MN-major)
// with p as two bf16 pieces (the first is p cut to 8 bits, the second the rest
// rounded: 2^-15), which take the scores' columns.  Two threads per row have 64 keys
// of a tile each; the reference m of a row moves only when a tile's largest score
// exceeds it by more than 8 (log2), and O is rescaled then: the halves exchange their
// maxima only when one of a row tile's rows has to move.
//
// Bound: the tensor core.  A tile of 128 keys takes 256 rows of 128 features 16
// products of 128 x 128 x 16 for S and 32 for PV (both pieces), 64 cycles each; its
// 32,768 exponentials take 2,048 cycles and shared memory 2,560 (S reads 2 x 8 x 8
// KB, PV 2 x 16 x 4 KB, TMA writes 64 KB, at 128 bytes a cycle).  The two row tiles
// alternate between the tensor core and the softmax: 4,100 cycles measured, 56 % of
// the tensor core over a launch.  3 sequences of 9,001 to 16,300 keys x 8 key heads x
// 252 rows: 58 us (104 with the rows along N); one thread per row with 128 scores in
// registers instead of two with 64: 61 and 63 us before the splits were balanced.
//
// Work: a CTA per (split, sequence, key head, block of 256 rows), key heads the
// fastest (they lie side by side in the cache).  Partials as in mha_rows.cu.
//
// Roles: four softmax warpgroups (two per row tile; they also load its Q and write
// its output), one MMA lane, one TMA lane.  Every wait is bounded.
#include <cuda_bf16.h>

#include "kernels.h"
#include "rows.cuh"

namespace mha {
namespace {

template <int W_>
struct BlockCfg {
  static constexpr int W = W_;                          // widest head: 64 or 128
  static constexpr int CHUNK = kKeys * 128;             // [128 rows x 64 features], 128-byte swizzle
  static constexpr int TILE = W / 64 * CHUNK;           // a tile of Q, K or V
  static constexpr int SLOTS = W == 64 ? 8 : 5;         // ring of K and V tiles
  static constexpr int THREADS = 640;
  static constexpr int OFF_Q = SLOTS * TILE;            // + row tile * TILE
  static constexpr int OFF_MISC = OFF_Q + 2 * TILE;
  static constexpr int OFF_XCHG = OFF_MISC + 256;       // a value per row [256]
  static constexpr int SMEM = OFF_XCHG + 1024 + 1024;
  static_assert(SMEM <= 232448, "shared memory");
  // barriers
  static constexpr int FULL = 0;             // + slot
  static constexpr int EMPTY = SLOTS;        // + slot
  static constexpr int Q_FULL = 2 * SLOTS;   // + row tile (eight warps)
  static constexpr int S_FULL = Q_FULL + 2;  // + row tile
  static constexpr int P_FULL = S_FULL + 2;  // + row tile (eight warps)
  static constexpr int O_DONE = P_FULL + 2;  // + row tile
  static constexpr int DRAIN = O_DONE + 2;
  static constexpr int NBAR = DRAIN + 1;
  static constexpr int OFF_TMEM = OFF_MISC + 8 * NBAR;
  static constexpr int OFF_ABORT = OFF_TMEM + 4;
  static constexpr int OFF_SHOWN = OFF_MISC + 224;      // drafted keys that some row sees (256 bits)
  static_assert(8 * NBAR + 8 <= 224, "barrier area");
  // TMEM: S_0 | S_1 (128 columns each, then P_g's two pieces) | O_0 | O_1
  static constexpr uint32_t TM_O = 256;
  static constexpr uint32_t TMEM_COLS = 512;
  // registers: a softmax thread holds 64 scores
  static constexpr int REGS_SOFT = 104, REGS_OTHER = 64;
  static_assert(REGS_SOFT * 512 + REGS_OTHER * 128 <= 96 * THREADS, "register split");
};

constexpr float kSlack = 8.f;  // a row's reference moves beyond this (log2)

// True for every thread of a row tile's two warpgroups when any of them passes true
// (named barrier `id` over their 256 threads).
__device__ __forceinline__ bool any_of_256(uint32_t id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "r"(id)
      : "memory");
  return r != 0;
}

// Which of 32 keys from `off` on, counted from the first drafted key, the row of
// drafted token t sees: all of the prefix (negative), the drafted ones by its mask
// words (or those up to t), none behind.
__device__ __forceinline__ uint32_t sees_32(const RowsParams& p, int b, int t, bool live, int off) {
  if (off <= -32) return ~0u;
  auto word = [&](int x) -> uint64_t {
    if (!live || x >= p.words) return 0;
    if (p.tree_mask) return __ldg(p.tree_mask + (static_cast<long long>(b) * p.T + t) * p.words + x);
    const int bits = t + 1 - 64 * x;
    return bits >= 64 ? ~0ull : (bits <= 0 ? 0ull : (1ull << bits) - 1);
  };
  if (off < 0) return ((1u << -off) - 1) | static_cast<uint32_t>(word(0) << -off);
  const int sh = off & 63;
  const uint64_t lo = word(off >> 6) >> sh;
  return static_cast<uint32_t>(sh <= 32 ? lo : lo | (word((off >> 6) + 1) << (64 - sh)));
}

template <int W>
__global__ void __launch_bounds__(BlockCfg<W>::THREADS, 1)
    rows_block_kernel(const __grid_constant__ RowsParams p) {
  using C = BlockCfg<W>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t s_base = smem_u32(smem);
  auto bar = [&](int i) { return s_base + C::OFF_MISC + 8 * i; };
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_TMEM);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
  uint32_t* shown = reinterpret_cast<uint32_t*>(smem + C::OFF_SHOWN);
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int tid = static_cast<int>(threadIdx.x);
  constexpr int kMmaWarp = 16, kLoadWarp = 17;

  if (tid == 0) {
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(bar(C::FULL + i), 1);
      mbar_init(bar(C::EMPTY + i), 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(bar(C::Q_FULL + g), 8);
      mbar_init(bar(C::S_FULL + g), 1);
      mbar_init(bar(C::P_FULL + g), 8);
      mbar_init(bar(C::O_DONE + g), 1);
    }
    mbar_init(bar(C::DRAIN), 1);
    for (int i = 0; i < 8; ++i) shown[i] = 0;
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), C::TMEM_COLS);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();  // global memory only from here on
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int n_rows = p.T * p.G;
  const int blocks = (n_rows + kBlockRows - 1) / kBlockRows;
  Unit it;
  {
    const int index = static_cast<int>(blockIdx.x), part = index / p.units;
    int b = part % p.B, split = part / p.B, per = 0;
    bool there = true;
    if (balanced(p)) {
      int first, splits;
      balance(p, lane, &first, &splits, &per);
      const unsigned has = __ballot_sync(0xffffffffu, part >= first && part < first + splits);
      there = has != 0;
      b = max(0, __ffs(has) - 1);
      split = part - __shfl_sync(0xffffffffu, first, b);
    }
    if (longest_first(p, kSms)) {
      const int place = place_of(p, lane);  // (by the whole warp)
      b = __ffs(__ballot_sync(0xffffffffu, lane < p.B && place == b)) - 1;
    }
    it = unit_of(p, index, blocks, b, split, per);
    if (!there) it.splits = 0;
  }
  const int n = it.t1 - it.t0;
  const int rows_here = min(kBlockRows, n_rows - it.rb * kBlockRows);
  const int tiles_m = rows_here > 128 ? 2 : 1;
  const bool works = it.splits > 0 && n > 0;  // (no such unit; no key at all)

  if (warp >= kMmaWarp) {
    regs_decrease<C::REGS_OTHER>();
    if (warp == kLoadWarp && works) {
      // ---- TMA producer (one lane): K(0) V(0) K(1) V(1) ...
      const int site = kRoleRowsLoad * 64;
      if (elect_one()) {
        const int chunks = (p.d + 63) / 64;
        int item = 0;
        bool ok = true;
        auto load = [&](const CUtensorMap* big, const CUtensorMap* small, int key) {
          const int s = item % C::SLOTS;
          ok = ok && (item < C::SLOTS || thread_wait(bar(C::EMPTY + s), ((item / C::SLOTS) - 1) & 1, abort_flag,
                                                     site + C::EMPTY + s));
          if (!ok) return;
          // whole in boxes of 128 keys, a ragged last tile in boxes of kBoxKeys as
          // far as it goes
          const int boxes = it.end - key >= kKeys ? 0 : (it.end - key + kBoxKeys - 1) / kBoxKeys;
          mbar_arrive_expect_tx(bar(C::FULL + s), chunks * 128 * (boxes == 0 ? kKeys : boxes * kBoxKeys));
          for (int c = 0; c < chunks; ++c) {
            const uint32_t dst = s_base + s * C::TILE + c * C::CHUNK;
            if (boxes == 0) {
              tma_load_4d(dst, big, bar(C::FULL + s), 64 * c, it.hk, key, it.b);
            } else {
              for (int x = 0; x < boxes; ++x)
                tma_load_4d(dst + x * kBoxKeys * 128, small, bar(C::FULL + s), 64 * c, it.hk, key + x * kBoxKeys,
                            it.b);
            }
          }
          ++item;
        };
        for (int x = it.t0; x < it.t1 && ok; ++x) {
          load(&p.tm_k, &p.tm_k_box, x * kKeys);
          load(&p.tm_v, &p.tm_v_box, x * kKeys);
        }
        // every copy started must land before the CTA exits
        volatile int never = 0;
        for (int x = max(0, item - C::SLOTS); x < item; ++x)
          mbar_wait(bar(C::FULL + x % C::SLOTS), (x / C::SLOTS) & 1, &never, p.status, site + x % C::SLOTS);
      }
      __syncwarp();
    } else if (warp == kMmaWarp && works) {
      // ---- MMA issuer (one lane)
      const int site = kRoleRowsMma * 64;
      if (elect_one()) {
        constexpr uint32_t idesc_s = idesc_bf16_f32(128, kKeys, false, false);
        constexpr uint32_t idesc_o = idesc_bf16_f32(128, W, false, true);
        const int n_ks = (p.d + 15) / 16;  // (what lies behind d is 0)
        const uint64_t dq0 = smem_desc_sw128(s_base + C::OFF_Q, 16, 1024);
        const uint64_t dk0 = smem_desc_sw128(s_base, 16, 1024);
        const uint64_t dv0 = smem_desc_sw128(s_base, C::CHUNK, 1024);
        bool ok = true;
        auto wait = [&](int id, uint32_t parity) { ok = ok && thread_wait(bar(id), parity, abort_flag, site + id); };
        // tile i's K lies in ring slot 2 i, its V in 2 i + 1 (modulo the ring)
        for (int i = -1; i < n && ok; ++i) {
          for (int g = 0; g < tiles_m && ok; ++g) {
            if (i >= 0) {
              // O_g += P_g V(i)
              const int item = 2 * i + 1, slot = item % C::SLOTS;
              wait(C::P_FULL + g, i & 1);
              wait(C::FULL + slot, (item / C::SLOTS) & 1);
              if (!ok) break;
              tc_fence_after();
              const uint64_t b = dv0 + static_cast<uint64_t>((slot * C::TILE) >> 4);
#pragma unroll
              for (int ks = 0; ks < 2 * (kKeys / 16); ++ks)  // (both pieces of p)
                umma_ts(tmem + C::TM_O + g * W, tmem + 128 * g + 8 * ks,
                        b + static_cast<uint64_t>((ks % (kKeys / 16) * 2048) >> 4), idesc_o,
                        (i > 0 || ks > 0) ? 1u : 0u);
              if (g == tiles_m - 1) umma_commit(bar(C::EMPTY + slot));
              if (i + 1 == n) umma_commit(bar(C::O_DONE + g));
            }
            if (i + 1 < n) {
              // S_g of the next tile, over P_g's columns (the tensor core works in order)
              const int item = 2 * i + 2, slot = item % C::SLOTS;
              if (i < 0) wait(C::Q_FULL + g, 0);
              wait(C::FULL + slot, (item / C::SLOTS) & 1);
              if (!ok) break;
              tc_fence_after();
              const uint64_t a = dq0 + static_cast<uint64_t>((g * C::TILE) >> 4);
              const uint64_t b = dk0 + static_cast<uint64_t>((slot * C::TILE) >> 4);
#pragma unroll
              for (int ks = 0; ks < W / 16; ++ks) {
                if (ks >= n_ks) break;
                const uint64_t off = static_cast<uint64_t>(((ks >> 2) * C::CHUNK + (ks & 3) * 32) >> 4);
                umma_ss(tmem + 128 * g, a + off, b + off, idesc_s, ks > 0 ? 1u : 0u);
              }
              umma_commit(bar(C::S_FULL + g));
              if (g == tiles_m - 1) umma_commit(bar(C::EMPTY + slot));
            }
          }
        }
        // every tensor-core operation issued must be complete before TMEM is freed
        umma_commit(bar(C::DRAIN));
        volatile int never = 0;
        mbar_wait(bar(C::DRAIN), 0, &never, p.status, site + C::DRAIN);
      }
      __syncwarp();
    }
  } else {
    regs_increase<C::REGS_SOFT>();
    // ---- softmax: two threads per row r of the unit, 64 keys of a tile each; row
    // tile g has the warpgroups g (first half) and g + 2
    const int g = (warp >> 2) & 1, half = warp >> 3, kt = tid & 127, r = 128 * g + kt;
    const int row = it.rb * kBlockRows + r;  // (drafted token, query head of the group)
    const bool exists = r < rows_here;
    const int t = exists ? row / p.G : 0;
    const long long out_row =
        (static_cast<long long>(it.b) * p.T + t) * p.H + it.hk * p.G + (exists ? row - t * p.G : 0);
    const bool live = exists && t < it.live;
    const int site = kRoleRowsSoftmax * 64;
    const uint32_t nbar = 1 + g;
    // op(first half's x, second half's x) for both threads of a row
    volatile float* between = reinterpret_cast<volatile float*>(smem + C::OFF_XCHG) + r;
    auto of_row = [&](float x, auto op) {
      if (half == 0) *between = x;
      named_barrier(nbar, 256);
      if (half == 1) *between = x = op(*between, x);
      named_barrier(nbar, 256);
      return half == 0 ? *between : x;
    };
    if (g < tiles_m && works) {
      bool ok = true;
      auto wait = [&](int id, uint32_t parity) { ok = ok && thread_wait(bar(id), parity, abort_flag, site + id); };
      // The mask words of the unit's rows together, for the tiles of drafted keys: a word
      // of every 64th token to a thread (asked for ahead of Q).
      uint64_t any = 0;
      if (g == 0 && p.tree_mask && it.t1 * kKeys > it.n && (tid & 3) < p.words) {
        const int first = it.rb * kBlockRows / p.G + ((kt + 128 * half) >> 2);
        const int last = min((it.rb * kBlockRows + rows_here - 1) / p.G, it.live - 1);
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (first + 64 * x <= last)
            any |= __ldg(p.tree_mask + (static_cast<long long>(it.b) * p.T + first + 64 * x) * p.words + (tid & 3));
      }
      // Q (zeros past the last row)
      {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + out_row * p.d);
        const uint32_t to = s_base + C::OFF_Q + g * C::TILE + kt * 128;
        constexpr int PER = W / 16;  // 16-byte pieces of a row per thread
        uint4 v[PER];
#pragma unroll
        for (int x = 0; x < PER; ++x) {
          v[x] = make_uint4(0, 0, 0, 0);
          if (exists && 8 * (half * PER + x) < p.d) v[x] = __ldg(src + half * PER + x);
        }
#pragma unroll
        for (int x = 0; x < PER; ++x) {
          const int y = half * PER + x;
          st_shared_v4(to + (y >> 3) * C::CHUNK + (((y & 7) ^ (kt & 7)) << 4), v[x].x, v[x].y, v[x].z, v[x].w);
        }
        fence_proxy_async_smem();
        warp_arrive(bar(C::Q_FULL + g), lane);
      }
      if (any) {
        // (the barrier of the first tile comes before these are read)
        atomicOr(shown + 2 * (tid & 3), static_cast<uint32_t>(any));
        atomicOr(shown + 2 * (tid & 3) + 1, static_cast<uint32_t>(any >> 32));
      }
      const float scale = p.scale_log2;  // (positive)
      const uint32_t t_lane = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      const uint32_t s_at = t_lane + 128 * g, o_at = t_lane + C::TM_O + g * W;
      float ref = 0.f, l0 = 0.f, l1 = 0.f;  // (the sums: of this thread's keys)
      bool seen = false;
      for (int i = 0; i < n; ++i) {
        const int key0 = (it.t0 + i) * kKeys;
        wait(C::S_FULL + g, i & 1);
        tc_fence_after();
        uint32_t s[2][32];
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_ld32(s_at + 64 * half + 32 * c, s[c]);
        tmem_ld_wait();
        if (key0 + kKeys > it.n) {
          // a tile that reaches behind the prefix
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int key = key0 + 64 * half + 32 * c;
            uint32_t sees = sees_32(p, it.b, t, live, key - it.n);
            if (key + 32 > it.end) sees = key >= it.end ? 0u : sees & ((1u << (it.end - key)) - 1);
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (!((sees >> x) & 1)) s[c][x] = __float_as_uint(-INFINITY);
          }
        }
        float top = -INFINITY, top1 = -INFINITY;
#pragma unroll
        for (int x = 0; x < 32; x += 2) {
          top = fmax3(top, __uint_as_float(s[0][x]), __uint_as_float(s[0][x + 1]));
          top1 = fmax3(top1, __uint_as_float(s[1][x]), __uint_as_float(s[1][x + 1]));
        }
        top = fmaxf(top, top1) * scale;
        const float limit = seen ? ref + kSlack : -INFINITY;
        // (this barrier also keeps P, which takes the scores' columns, behind the
        // other half's reading of them)
        tc_fence_before();
        const bool moves = any_of_256(nbar, top > limit);
        tc_fence_after();
        if (moves) {
          top = of_row(top, [](float x, float y) { return fmaxf(x, y); });
          const bool rise = top > limit;
          // (what a row without a key so far has in O is 0 at any reference)
          const float f = rise && seen ? ex2_approx(ref - top) : 1.f;
          if (rise) {
            ref = top;
            seen = true;
            l0 *= f;
            l1 *= f;
          }
          // (the scores were issued behind the last product, so O is complete)
          if (i > 0 && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
            for (int c = half * (W / 2); c < (half + 1) * (W / 2); c += 16) {
              uint32_t o[16];
              tmem_ld16(o_at + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
              tmem_st16(o_at + c, o);
            }
          }
        }
        const float nref = -ref;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t w1[16], w2[16];
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            float p0, p1, y0, y1;
            fma2(p0, p1, __uint_as_float(s[c][x]), __uint_as_float(s[c][x + 1]), scale, scale, nref, nref);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            add2(l0, l1, l0, l1, p0, p1);
            // the first piece is cut, not rounded: its bits are p's own
            const uint32_t u0 = __float_as_uint(p0) & 0xffff0000u, u1 = __float_as_uint(p1) & 0xffff0000u;
            w1[x >> 1] = __byte_perm(u0, u1, 0x7632);
            fma2(y0, y1, __uint_as_float(u0), __uint_as_float(u1), -1.f, -1.f, p0, p1);
            w2[x >> 1] = pack_bf16x2(y0, y1);
          }
          tmem_st16(s_at + 32 * half + 16 * c, w1);
          tmem_st16(s_at + 64 + 32 * half + 16 * c, w2);
        }
        if (g == 0 && key0 + kKeys > it.n) {
          // V rows that no row of the unit sees may hold anything, and 0 * NaN would be
          // NaN: those past the last key, and drafted ones whose bit no row sets; the
          // second row tile's product comes later
          const int key = key0 + kt, j = key - it.n;
          const bool hidden = key >= it.end || (p.tree_mask && j >= 0 && !((shown[j >> 5] >> (j & 31)) & 1));
          if (__any_sync(0xffffffffu, hidden)) {
            const int item = 2 * i + 1, slot = item % C::SLOTS;
            wait(C::FULL + slot, (item / C::SLOTS) & 1);
            if (hidden) {
#pragma unroll 1
              for (int x = half * (W / 16); x < (half + 1) * (W / 16); ++x)
                st_shared_v4(s_base + slot * C::TILE + (x >> 3) * C::CHUNK + kt * 128 + (x & 7) * 16, 0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(bar(C::P_FULL + g), lane);
      }

      // ---- epilogue
      wait(C::O_DONE + g, 0);
      tc_fence_after();
      const bool good = ok && *abort_flag == 0;
      const float sum = of_row(l0 + l1, [](float x, float y) { return x + y; });
      const float L = live && good ? sum : 0.f;
      const bool whole = it.splits == 1;
      const float a = L > 0.f ? (whole ? 1.f / L : 1.f) : 0.f;
      const long long part = static_cast<long long>(it.part - it.b) * p.T * p.H + out_row;
      if (exists && half == 0) {
        if (!whole) {
          p.part_m[part] = L > 0.f ? ref : -INFINITY;
          p.part_l[part] = L;
        } else if (p.lse) {
          p.lse[(static_cast<long long>(it.b) * p.H + it.hk * p.G + (row - t * p.G)) * p.T + t] =
              L > 0.f ? (ref + __log2f(L)) * 0.69314718055994531f : -INFINITY;
        }
      }
#pragma unroll 1
      for (int c = half * (W / 2); c < (half + 1) * (W / 2); c += 16) {
        uint32_t o[16];
        tmem_ld16(o_at + c, o);
        tmem_ld_wait();
        if (!exists || c >= p.d) continue;
#pragma unroll
        for (int x = 0; x < 16; ++x) o[x] = a > 0.f ? __float_as_uint(__uint_as_float(o[x]) * a) : 0u;
        if (whole) {
          uint32_t y[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) y[x] = pack_bf16x2(__uint_as_float(o[2 * x]), __uint_as_float(o[2 * x + 1]));
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + out_row * p.d + c);
          dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
          if (c + 8 < p.d) dst[1] = make_uint4(y[4], y[5], y[6], y[7]);  // (d is a multiple of 8)
        } else {
          uint4* dst = reinterpret_cast<uint4*>(p.part_o + part * W + c);
#pragma unroll
          for (int x = 0; x < 4; ++x) dst[x] = make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
        }
      }
      tc_fence_before();
    } else if (it.splits > 0 && n == 0 && exists && half == 0) {
      // no key at all: output 0, log-sum-exp -inf
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + out_row * p.d);
      for (int x = 0; 8 * x < p.d; ++x) dst[x] = make_uint4(0, 0, 0, 0);
      if (p.lse)
        p.lse[(static_cast<long long>(it.b) * p.H + it.hk * p.G + (row - t * p.G)) * p.T + t] = -INFINITY;
    }
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
  if (tid == 0 && *abort_flag != 0 && atomicCAS(&p.status->code, 0, 7 /* MHA_ERR_TIMEOUT */) == 0) {
    p.status->site = *abort_flag - 1;
    p.status->block = static_cast<int>(blockIdx.x);
  }
}

template <int W>
cudaError_t launch_block_cfg(const RowsParams& p, cudaStream_t stream, LaunchInfo* info) {
  using C = BlockCfg<W>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static bool attr_set[64] = {};
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(rows_block_kernel<W>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  const dim3 grid(static_cast<unsigned>(p.B * p.units * p.n_splits));
  e = launch_serialized(rows_block_kernel<W>, grid, dim3(C::THREADS), C::SMEM, stream, p);
  if (e != cudaSuccess) return e;
  if (info) {
    info->kernels = 1;
    info->grid = static_cast<int>(grid.x);
    info->block = C::THREADS;
    info->smem = C::SMEM;
  }
  return e;
}

}  // namespace

cudaError_t launch_rows_block(const RowsParams& p, cudaStream_t stream, LaunchInfo* info) {
  return p.d <= 64 ? launch_block_cfg<64>(p, stream, info) : launch_block_cfg<128>(p, stream, info);
}

}  // namespace mha

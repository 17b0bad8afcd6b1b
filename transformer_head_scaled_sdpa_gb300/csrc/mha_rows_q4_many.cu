// mha_rows_q4_many.cu -- attention of many query rows per key head over the 4-bit
// key/value cache, on the 5th-generation tensor cores, sm_103a: more than sixteen rows
// (32 of heads up to 64 features); fewer are mha_rows_q4.cu's, whose formulas these are.
//
// With rows enough, arithmetic bounds the step, and both products go to tcgen05, keys (then
// features) along the 128 rows of its tile and the query rows along its columns:
//   S^T [128 keys x NR] = K Q^T       A: K in tensor memory, a lane per key
//   O^T [features x NR] += V^T P^T    A: V in shared memory, read transposed; B: weights
// Codes become fp16 subnormals (c 2^-24, exact; odd ones 16 times too large) on the way
// there: a thread has a key, takes its packed row from the ring that TMA fills, masks and
// shifts, and writes keys to tensor memory (tcgen05.st) and values to shared memory in the
// layout that a 128-byte swizzled TMA tile would have.  A word's eight codes come out in
// the order 0 4 1 5 2 6 3 7; Q is laid out in it, and the output's rows are read in it.
// In tensor memory K costs neither shared memory's room nor its bandwidth; V, whose rows
// are keys and whose lanes would have to be features, would need a transposition there.
//
// Softmax: a thread has a key, that is its offset and step, and RPT of the rows; what a
// row needs (its factors and reference) is read by all lanes at once.  Rows of like sizes
// share a power of two in Q, and the factor of their products (8 x 24 heads x 56 rows of 128
// features x 2,048 to 4,096 keys 68 us, 74 with a factor each); a row that is far larger, or
// infinite, must not take the others' digits, and then each has its own.  Weights are rounded to
// fp16 (2^-11 relative); scores and sums are float32 (rows_q4.cuh: what sums of products cut);
// the denominator and the offsets' sum stay in a thread's registers
// until the unit ends.  References move for all keys of a tile, by a vote of the
// warpgroup, when a weight would pass 2^kLimit; O is then scaled in tensor memory.
//
// Roles: softmax warps (8, or 16), four warps that unpack keys, four that unpack values
// (one group for both: 58 us when this took 49, 8 x 12 heads x 32 rows of 256 features x 2,048
// to 4,096 keys), one that issues the MMAs, one that loads.  Scores and weights have two
// buffers each, S(t + 1) is formed before PV(t).  The MMA warp runs converged and elects a
// lane to issue, which keeps descriptors in uniform registers: issued by one lane on its own
// an MMA took 150 cycles (32 rows of 128 features 64 us when this took 45).
//
// What bounds it: the softmax warps, 1,900 to 2,400 cycles a tile (scores read and scaled
// 900, vote and waits 500, weights 450), with one CTA to an SM, and 15 to 20 thousand
// cycles that a unit costs beside its tiles (its lengths 2,600, Q 4,500, first tile 5,000,
// sums and outputs 5,000).  5 x 2 key heads x 56 rows of 256 features x 7,001 to 20,000
// keys: 33.4 us (5 of them the merge of splits), 47 on mma.sync in units of 16 rows; 8 x
// 24 heads x 56 rows of 128 features x 2,048 to 4,096 keys 68 against 95, 252 rows 232
// against 350.
#include <cuda_bf16.h>

#include <type_traits>

#include "rows_q4.cuh"

namespace mha {
namespace {

constexpr int kRoleMany = 21;

// W: widest head; NR: rows of a unit.
template <int W_, int NR_, int RPT_, int VST_, int SLOTS_>
struct ManyCfg {
  static constexpr int W = W_, NR = NR_;
  static constexpr int ROW = W / 2, TILE = kKeys * ROW;  // packed bytes of a row, of a tile's keys or values
  static constexpr int KC = W / 32;                      // 16-byte pieces of a row
  static constexpr int BLKS = W == 256 ? 2 : 1, FB = W / BLKS;  // blocks of features of the output
  static constexpr int CHUNK = kKeys * 128;              // [128 keys x 64 features] in fp16, 128-byte swizzle
  static constexpr int VBYTES = FB / 64 * CHUNK;
  static constexpr int KST = 2, VST = VST_;              // unpacked keys (tensor memory), blocks of values
  static constexpr int SLOTS = SLOTS_;                   // packed tiles
  static constexpr int RPT = RPT_, WGS = NR / RPT;         // rows of a softmax thread, softmax warpgroups
  static constexpr int Q_BYTES = NR * W * 2, P_BYTES = kKeys * NR * 2;
  static constexpr uint32_t TM_K = 0, TM_S = KST * (W / 2), TM_O = TM_S + 2 * NR;
  static constexpr uint32_t TM_USED = TM_O + BLKS * NR;
  static constexpr uint32_t TMEM_COLS = TM_USED <= 128 ? 128 : (TM_USED <= 256 ? 256 : 512);
  static_assert(TM_USED <= 512 && NR % RPT == 0, "tensor memory");
  static constexpr int OFF_RING = VST * VBYTES;
  static constexpr int OFF_Q = OFF_RING + SLOTS * TILE;
  static constexpr int OFF_P = OFF_Q + Q_BYTES;
  static constexpr int OFF_SCALES = OFF_P + 2 * P_BYTES;        // a warpgroup's words
  static constexpr int OFF_MASKS = OFF_SCALES + WGS * Scales::BYTES;  // uint64 [NR][4]
  // float4 [NR / 2]: of two rows, the factors of offsets, and what is added to scores; then
  // float [NR]: of products
  static constexpr int OFF_FACTORS = OFF_MASKS + NR * 32;
  static constexpr int OFF_ROWS = OFF_FACTORS + NR * 12;        // float [5][NR], int [NR]
  static constexpr int OFF_RED = OFF_ROWS + NR * 24;            // float [2][NR][4]
  // barriers
  static constexpr int FULL_K = 0, FULL_V = SLOTS, EMPTY = 2 * SLOTS;  // + slot
  static constexpr int K_FULL = 3 * SLOTS, K_EMPTY = K_FULL + KST;  // + stage
  static constexpr int V_FULL = K_EMPTY + KST, V_EMPTY = V_FULL + VST;
  static constexpr int Q_FULL = V_EMPTY + VST, S_FULL = Q_FULL + 1;  // + tile & 1
  static constexpr int P_FULL = S_FULL + 2;  // + tile & 1
  static constexpr int BUT_LAST = P_FULL + 2, DRAIN = BUT_LAST + 1;  // the products of all tiles but the last, of all
  static constexpr int NBAR = DRAIN + 1;
  static constexpr int OFF_UNIT = OFF_RED + NR * 32;
  static constexpr int OFF_BAR = OFF_UNIT + static_cast<int>(sizeof(Unit));
  static constexpr int OFF_TMEM = OFF_BAR + 8 * NBAR, OFF_ABORT = OFF_TMEM + 4;
  static constexpr int SMEM = OFF_ABORT + 4 + 1024;
  static constexpr int SOFT = 4 * WGS, UNPACK = 4;  // warps (for keys, and for values); then MMA, loads, two idle
  static constexpr int THREADS = 32 * (SOFT + 2 * UNPACK + 4);
  // registers: the softmax warps take from the others
  static constexpr int REGS = 65536 / THREADS / 8 * 8, REGS_OTHER = WGS == 4 ? 40 : 48;
  static constexpr int REGS_SOFT = (REGS * THREADS - REGS_OTHER * (THREADS - 32 * SOFT)) / (32 * SOFT) / 8 * 8;
  static_assert(SMEM <= 232448 && OFF_BAR % 8 == 0 && OFF_MASKS % 16 == 0, "shared memory");
};

// Instruction descriptor of kind::f16 with fp16 operands (fields as idesc_bf16_f32).
constexpr uint32_t idesc_f16_f32(int M, int N, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | (static_cast<uint32_t>(a_mn_major) << 15) | (static_cast<uint32_t>(b_mn_major) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// A word's eight codes as fp16: codes 0 and 4, 1 and 5 (16 times too large), 2 and 6, 3
// and 7 (16 times).
__device__ __forceinline__ void unpack(uint32_t w, uint32_t* r) {
  r[0] = w & 0x000f000fu;
  r[1] = w & 0x00f000f0u;
  r[2] = (w >> 8) & 0x000f000fu;
  r[3] = (w >> 8) & 0x00f000f0u;
}
// Feature (of eight) at place x of that order.
__device__ __forceinline__ int feature_at(int x) { return (x >> 1) + 4 * (x & 1); }

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) rows_q4_many_kernel(const __grid_constant__ RowsParams p) {
  constexpr int W = C::W, NR = C::NR;
  constexpr int KC = C::KC, RPT = C::RPT, BLKS = C::BLKS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t base = smem_u32(smem);
  auto bar = [&](int id) { return base + C::OFF_BAR + 8u * static_cast<uint32_t>(id); };
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_TMEM);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  constexpr int kMmaWarp = C::SOFT + 2 * C::UNPACK, kLoadWarp = kMmaWarp + 1;
  if (tid == 0) {
    for (int s = 0; s < C::SLOTS; ++s) {
      mbar_init(bar(C::FULL_K + s), 1);
      mbar_init(bar(C::FULL_V + s), 1);
      mbar_init(bar(C::EMPTY + s), C::UNPACK);
    }
    for (int s = 0; s < C::KST; ++s) {
      mbar_init(bar(C::K_FULL + s), C::UNPACK);
      mbar_init(bar(C::K_EMPTY + s), 1);
    }
    for (int s = 0; s < C::VST; ++s) {
      mbar_init(bar(C::V_FULL + s), C::UNPACK);
      mbar_init(bar(C::V_EMPTY + s), 1);
    }
    mbar_init(bar(C::Q_FULL), C::SOFT);
    mbar_init(bar(C::S_FULL), 1);
    mbar_init(bar(C::S_FULL + 1), 1);
    mbar_init(bar(C::P_FULL), C::SOFT);
    mbar_init(bar(C::P_FULL + 1), C::SOFT);
    mbar_init(bar(C::BUT_LAST), 1);
    mbar_init(bar(C::DRAIN), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), C::TMEM_COLS);
    tmem_relinquish();
    tc_fence_before();
  }
  griddep_wait();
  // (one warp finds the unit: all 28 at it were 1,500 cycles of each other's instructions)
  const int n_rows = p.T * p.G;
  Unit* unit = reinterpret_cast<Unit*>(smem + C::OFF_UNIT);
  if (warp == 0) {
    Unit u = {};
    const bool has = this_unit(p, (n_rows + NR - 1) / NR, kSms, lane, &u);
    u.pad[0] = has;
    if (lane == 0) *unit = u;
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // (the next launch's CTAs take tensor memory too: only now that this one has its own)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const Unit it = *unit;
  const bool mine = it.pad[0] != 0;
  const int first = it.t0 * kKeys, stop = mine ? min(it.t1 * kKeys, it.end) : 0;
  const int tiles = stop > first ? (stop - first + kKeys - 1) / kKeys : 0;
  const RingItems items{C::SLOTS, tiles};
  auto site = [&](int id) { return kRoleMany * 64 + id; };

  if (warp >= C::SOFT) {
    regs_decrease<C::REGS_OTHER>();
    if (!mine) {
      // (more units than the sequences have splits)
    } else if (warp == kLoadWarp) {
      // ---- items K0 K1 V0 K2 V1 ... of packed codes
      if (lane == 0) {
        const Loader<W> load{p, it, stop};
        bool ok = true;
        int x = 0;
        SlotParity keys, values;  // of what was sent
        for (; x < 2 * tiles; ++x) {
          const int slot = items.slot(x);
          if (x >= C::SLOTS)
            ok = thread_wait(bar(C::EMPTY + slot), (x / C::SLOTS - 1) & 1, abort_flag, site(C::EMPTY + slot));
          if (!ok) break;
          const bool v = items.is_values(x);
          const int key = first + items.tile(x) * kKeys, full = (v ? C::FULL_V : C::FULL_K) + slot;
          if (v) values.next(slot);
          else keys.next(slot);
          mbar_arrive_expect_tx(bar(full), load.bytes(key));
          load.copy(base + C::OFF_RING + slot * C::TILE, bar(full), key, v);
        }
        // the copies in flight must land before the CTA exits, also where a wait ran out
        volatile int never = 0;
        for (int y = max(0, x - C::SLOTS); y < x; ++y) {
          const int slot = items.slot(y);
          const bool v = items.is_values(y);  // (the slot's last item, and so the last of its barrier)
          const int full = (v ? C::FULL_V : C::FULL_K) + slot;
          mbar_wait(bar(full), v ? values.last(slot) : keys.last(slot), &never, p.status, site(full));
        }
      }
      __syncwarp();
    } else if (warp == kMmaWarp) {
      // ---- S(0), S(1), PV(0), S(2), PV(1), ...: the warp runs together, so that descriptors stay in
      // uniform registers, and one lane issues (all of it by one lane: 150 cycles an MMA)
      constexpr uint32_t idesc_s = idesc_f16_f32(128, NR, false, false);
      constexpr uint32_t idesc_o = idesc_f16_f32(C::FB, NR, true, true);
      const uint64_t dq = smem_desc_plain(base + C::OFF_Q, NR * 16, 128);
      const uint64_t dv = smem_desc_sw128(base, C::CHUNK, 1024);
      const uint64_t dp = smem_desc_plain(base + C::OFF_P, 128, kKeys * 16);
      bool ok = true;
      auto wait = [&](int id, int parity) {
        ok = ok && warp_wait(bar(id), parity & 1, abort_flag, site(id));
        tc_fence_after();
        return ok;
      };
      if (tiles > 0) wait(C::Q_FULL, 0);
#pragma unroll 1
      for (int t = 0; t <= tiles && tiles > 0 && ok; ++t) {
        if (t < tiles) {
          // (the scores of tile t - 2 are read: its weights were there for its values' products)
          const int st = t % C::KST;
          if (!wait(C::K_FULL + st, t / C::KST)) break;
          const uint32_t d = tmem + C::TM_S + (t & 1) * NR, a = tmem + C::TM_K + st * (W / 2);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < W / 16; ++k)  // (features past d are 0 on both sides)
              umma_ts(d, a + 8 * k, dq + static_cast<uint64_t>(2 * NR * k), idesc_s, k > 0 ? 1u : 0u);
            umma_commit(bar(C::S_FULL + (t & 1)));
            umma_commit(bar(C::K_EMPTY + st));
          }
          __syncwarp();
        }
        if (t > 0) {
          const int b = (t - 1) & 1;
          if (!wait(C::P_FULL + b, (t - 1) >> 1)) break;
#pragma unroll
          for (int blk = 0; blk < BLKS; ++blk) {
            const int x = (t - 1) * BLKS + blk, st = x % C::VST;
            if (!wait(C::V_FULL + st, x / C::VST)) break;
            const uint64_t a = dv + static_cast<uint64_t>((st * C::VBYTES) >> 4);
            const uint64_t w = dp + static_cast<uint64_t>((b * C::P_BYTES) >> 4);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < kKeys / 16; ++k)
                umma_ss(tmem + C::TM_O + blk * NR, a + static_cast<uint64_t>((k * 2048) >> 4),
                        w + static_cast<uint64_t>((k * 256) >> 4), idesc_o, (t > 1 || k > 0) ? 1u : 0u);
              umma_commit(bar(C::V_EMPTY + st));
              if (blk == BLKS - 1 && t == tiles - 1) umma_commit(bar(C::BUT_LAST));
            }
            __syncwarp();
          }
        }
      }
      // every tensor-core operation issued must be complete before TMEM is freed
      if (elect_one()) umma_commit(bar(C::DRAIN));
      __syncwarp();
      volatile int never = 0;
      mbar_wait(bar(C::DRAIN), 0, &never, p.status, site(C::DRAIN));
    } else if (warp < kMmaWarp) {
      // ---- unpacking: a thread has a key
      const int key = 32 * (warp & 3) + lane;
      const uint32_t packed = base + C::OFF_RING + key * C::ROW;
      const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
      bool ok = true;
      SlotParity landed;  // of this group's items
      auto wait = [&](int id, int parity) {
        ok = ok && warp_wait(bar(id), parity & 1, abort_flag, site(id));
        return ok;
      };
      auto words = [&](int slot, int c) { return ld_shared_v4(packed + slot * C::TILE + 16 * (c ^ swizzle<W>(key))); };
      auto keys = [&](int t) {
        const int slot = items.slot(items.keys(t)), st = t % C::KST;
        if (!wait(C::FULL_K + slot, landed.next(slot))) return;
        if (t >= C::KST && !wait(C::K_EMPTY + st, t / C::KST - 1)) return;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          const uint4 w = words(slot, c);
          uint32_t r[16];
          unpack(w.x, r);
          unpack(w.y, r + 4);
          unpack(w.z, r + 8);
          unpack(w.w, r + 12);
          tmem_st16(tmem + lanes + C::TM_K + st * (W / 2) + 16 * c, r);
        }
        warp_arrive(bar(C::EMPTY + slot), lane);
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(bar(C::K_FULL + st), lane);
      };
      auto values = [&](int t) {
        const int slot = items.slot(items.values(t));
        if (!wait(C::FULL_V + slot, landed.next(slot))) return;
#pragma unroll
        for (int blk = 0; blk < BLKS; ++blk) {
          const int y = t * BLKS + blk, st = y % C::VST;
          if (y >= C::VST && !wait(C::V_EMPTY + st, y / C::VST - 1)) return;
          const uint32_t to = base + st * C::VBYTES + key * 128;
#pragma unroll
          for (int c = 0; c < KC / BLKS; ++c) {
            const uint4 w = words(slot, blk * (KC / BLKS) + c);
            const uint32_t z[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t r[4];
              unpack(z[i], r);
              const int piece = 4 * c + i;
              st_shared_v4(to + (piece >> 3) * C::CHUNK + (((piece & 7) ^ (key & 7)) << 4), r[0], r[1], r[2], r[3]);
            }
          }
          fence_proxy_async_smem();
          if (blk == BLKS - 1) warp_arrive(bar(C::EMPTY + slot), lane);
          warp_arrive(bar(C::V_FULL + st), lane);
        }
      };
      if (warp < C::SOFT + C::UNPACK) {
        for (int t = 0; t < tiles && ok; ++t) keys(t);
      } else {
        for (int t = 0; t < tiles && ok; ++t) values(t);
      }
    }
  } else {
    regs_increase<C::REGS_SOFT>();
    if (mine) {
      // ---- softmax: a thread has a key and RPT of the rows
      const int wg = warp >> 2, w4 = warp & 3, kt = tid & 127, r0 = wg * RPT, nbar = 1 + wg;
      const int rows_here = min(max(n_rows - it.rb * NR - r0, 0), RPT);
      float4* factors = reinterpret_cast<float4*>(smem + C::OFF_FACTORS);
      auto less = [&](int r) { return reinterpret_cast<float*>(factors + r / 2) + 2 + (r & 1); };
      float* row_scale = reinterpret_cast<float*>(factors + NR / 2);
      float* row_ref = reinterpret_cast<float*>(smem + C::OFF_ROWS);  // references less kLift
      float* row_by = row_ref + NR;                                   // a move's factors, and differences
      float* row_down = row_by + NR;
      float* row_inv = row_down + NR;
      float* row_add = row_inv + NR;
      int* row_out = reinterpret_cast<int*>(row_add + NR);
      float* red = reinterpret_cast<float*>(smem + C::OFF_RED);       // [row][warp], of the second sum behind
      uint64_t(*masks)[4] = reinterpret_cast<uint64_t(*)[4]>(smem + C::OFF_MASKS);
      // Output row of row r of the unit (-1 past the last), t: its drafted token.
      auto out_row = [&](int r, int* t) {
        const int gr = it.rb * NR + r;
        *t = -1;
        if (gr >= n_rows) return -1;
        *t = p.G == 1 ? gr : gr / p.G;
        return (it.b * p.T + *t) * p.H + it.hk * p.G + (gr - *t * p.G);
      };
      const long long scales = (static_cast<long long>(it.b) * p.H_kv + it.hk) * p.Lk;
      const Scales words{base + C::OFF_SCALES + wg * Scales::BYTES + 8 * kt,
                         reinterpret_cast<const uint32_t*>(p.k_scale) + scales,
                         reinterpret_cast<const uint32_t*>(p.v_scale) + scales, kt, stop};
      words.start(first);
      constexpr int kNone = 1000;
      int common = kNone;  // the e of all rows
      float key_scale, factor_scale;
      {
        // Q: eight features to a lane, W / 8 lanes to a row
        constexpr int LPR = W / 8, RPW = 32 / LPR, PASSES = (NR + C::SOFT * RPW - 1) / (C::SOFT * RPW);
        static_assert(C::SOFT * RPW <= NR, "a row to every group of lanes");
        const int piece = lane % LPR;
        uint4 v[PASSES];
        int outs[PASSES];
#pragma unroll
        for (int y = 0; y < PASSES; ++y) {
          int t;
          outs[y] = out_row((y * C::SOFT + warp) * RPW + lane / LPR, &t);
          v[y] = make_uint4(0, 0, 0, 0);
          if (outs[y] >= 0 && t < it.live && 8 * piece < p.d)
            v[y] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                        static_cast<long long>(outs[y]) * p.d + 8 * piece));
        }
        const uint64_t bits = tid < NR * 4 ? mask_word(p, it, tid, out_row) : 0;
        // q 2^-e with the row's largest magnitude in [2^14, 2^15); where the unit's rows are within
        // 2^8 of one another (those of zeros aside) with the largest row's e, and one factor for all:
        // an fp16 of q is then off by up to 2^-27 of its row's largest (2^-31 in even features)
        int e[PASSES], top = -200, low = 200;
#pragma unroll
        for (int y = 0; y < PASSES; ++y) {
          const uint32_t x[4] = {v[y].x, v[y].y, v[y].z, v[y].w};
          float amax = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(x[i])), fabsf(bf16_hi(x[i]))));
#pragma unroll
          for (int z = 1; z < LPR; z <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, z));
          e[y] = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 14, -100);
          if (amax != 0.f) {
            if (amax < INFINITY) top = max(top, e[y]);
            low = min(low, amax < INFINITY ? e[y] : -300);  // (an infinity: no common factor)
          }
        }
        top = __reduce_max_sync(0xffffffffu, top);
        low = __reduce_min_sync(0xffffffffu, low);
        if (lane == 0) *reinterpret_cast<int2*>(red + 2 * warp) = make_int2(top, low);
        named_barrier(8, 32 * C::SOFT);
#pragma unroll
        for (int w = 0; w < C::SOFT; ++w) {
          const int2 z = *reinterpret_cast<const int2*>(red + 2 * w);
          top = max(top, z.x);
          low = min(low, z.y);
        }
        if (low <= top && top - low <= 8) common = top;
        const int shift = factor_shift(top, p.scale_log2);
        key_scale = pow2i(shift);
        factor_scale = pow2i(-shift) * p.scale_log2;
#pragma unroll
        for (int y = 0; y < PASSES; ++y) {
          const int r = (y * C::SOFT + warp) * RPW + lane / LPR;
          const uint32_t x[4] = {v[y].x, v[y].y, v[y].z, v[y].w};
          if (common != kNone) e[y] = common;
          const float inv = pow2i(-e[y]);
          float f[8], sum = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(x[i]) * inv;
            f[2 * i + 1] = bf16_hi(x[i]) * inv;
            sum += f[2 * i] + f[2 * i + 1];
          }
#pragma unroll
          for (int z = 1; z < LPR; z <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, z);
          st_shared_v4(base + C::OFF_Q + piece * (NR * 16) + r * 16, pack_f16x2(f[0], f[4]),
                       pack_f16x2(f[1] * 0.0625f, f[5] * 0.0625f), pack_f16x2(f[2], f[6]),
                       pack_f16x2(f[3] * 0.0625f, f[7] * 0.0625f));
          if (piece == 0) {
            const float scale = pow2i(e[y]) * factor_scale;
            reinterpret_cast<float*>(factors + r / 2)[r & 1] = scale * sum;
            row_scale[r] = scale * 16777216.f;  // (codes are 2^-24)
            *less(r) = 0.f;
            row_ref[r] = kNoRef;
            row_out[r] = outs[y];
          }
        }
        if (tid < NR * 4) masks[tid >> 2][tid & 3] = bits;
        fence_proxy_async_smem();
        warp_arrive(bar(C::Q_FULL), lane);
        named_barrier(8, 32 * C::SOFT);
      }
      const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * w4) << 16);
      float l[RPT], ofs[RPT];
#pragma unroll
      for (int r = 0; r < RPT; ++r) l[r] = ofs[r] = 0.f;
      const float scale_all = common != kNone ? pow2i(common) * factor_scale * 16777216.f : 0.f;
      bool ok = true, pending = true;  // a row has no reference yet
      auto wait = [&](int id, int parity) {
        ok = warp_wait(bar(id), parity & 1, abort_flag, site(id)) && ok;
        tc_fence_after();
      };
      // The products of all tiles before t, whose scores have been waited for: they come before the
      // scores of t + 1, whose commit covers them.  (A barrier for each tile's products, waited for at
      // these moves alone, would pass unseen phases, which a wait by parity cannot tell apart.)
      auto products_before = [&](int t) {
        if (t > 0) {
          if (t + 1 < tiles) wait(C::S_FULL + ((t + 1) & 1), (t + 1) >> 1);
          else wait(C::BUT_LAST, 0);
        }
      };
      // a live row of this thread to look after
      int own_t = -1;
      const bool own_live = kt < rows_here && out_row(r0 + kt, &own_t) >= 0 && own_t < it.live;
      uint2 kv = words.get(0, first);
#pragma unroll 1
      for (int t = 0; t < tiles; ++t) {
        const int tile0 = first + t * kKeys;
        const KeyFactors mine_f = key_factors(kv.x, kv.y, key_scale);
        wait(C::S_FULL + (t & 1), t >> 1);
        float x[RPT];
        {
          uint32_t raw[RPT];
          if constexpr (RPT == 32) tmem_ld32(lanes + C::TM_S + (t & 1) * NR + r0, raw);
          else tmem_ld16(lanes + C::TM_S + (t & 1) * NR + r0, raw);
          tmem_ld_wait();
          // x = S factor step + (factor' lo + (log2 stepv - m))
          auto scores = [&](auto own) {
            const float all = scale_all * mine_f.step;
#pragma unroll
            for (int r = 0; r < RPT; r += 2) {
              const float4 f = factors[(r0 + r) / 2];
              float u0, u1, a0 = all, a1 = all;
              add2(u0, u1, f.z, f.w, mine_f.v_log, mine_f.v_log);
              fma2(u0, u1, f.x, f.y, mine_f.lo, mine_f.lo, u0, u1);
              if constexpr (own) {
                const float2 a = *reinterpret_cast<const float2*>(row_scale + r0 + r);
                mul2(a0, a1, a.x, a.y, mine_f.step, mine_f.step);
              }
              fma2(x[r], x[r + 1], __uint_as_float(raw[r]), __uint_as_float(raw[r + 1]), a0, a1, u0, u1);
            }
          };
          if (common != kNone) scores(std::false_type{});
          else scores(std::true_type{});
        }
        float top = -INFINITY;
        if (tile0 + kKeys > min(it.n, stop)) {
          const KeyMask mask(tile0 + kt, stop, it.n);
#pragma unroll
          for (int r = 0; r < RPT; ++r) x[r] = mask.seen_by(masks, r0 + r) ? x[r] : -INFINITY;
        }
#pragma unroll
        for (int r = 0; r < RPT; r += 2) top = fmax3(top, x[r], x[r + 1]);
        if (any_of_128(nbar, pending || top > kLimit)) {
          // references up to this tile's maxima, what was summed down by as much
#pragma unroll
          for (int r = 0; r < RPT; ++r) {
            const float m = warp_max(x[r]);
            if (lane == 0) red[(r0 + r) * 4 + w4] = m;
          }
          named_barrier(nbar, 128);
          float ref = 0.f;
          if (kt < RPT) {
            const int r = r0 + kt;
            const float4 m4 = *reinterpret_cast<const float4*>(red + r * 4);
            const float m = fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w)), old = row_ref[r], sub = -*less(r);
            ref = m == -INFINITY ? old : fmaxf(old, m + sub - kLift);
            const float now = ref == kNoRef ? 0.f : ref;
            float down = sub - now;
            // (where references are so large that their places are not far below kLift, m must come
            // to lie in the weights' range all the same: the distance is then m's own)
            if (m + down > kLimit || (ref > old && m + down < 0.f)) down = -lifted(m);
            row_by[r] = old == kNoRef ? 1.f : ex2_approx(down);  // (nothing is summed up yet)
            row_down[r] = down;
            *less(r) = -now;
            row_ref[r] = ref;
          }
          pending = any_of_128(nbar, own_live && ref == kNoRef);
          products_before(t);
#pragma unroll
          for (int r = 0; r < RPT; ++r) {
            const float by = row_by[r0 + r];
            x[r] += row_down[r0 + r];
            l[r] *= by;
            ofs[r] *= by;
          }
          if (t > 0) {
#pragma unroll 1
            for (int blk = 0; blk < BLKS; ++blk)
#pragma unroll 1
              for (int g = 0; g < RPT; g += 16) {
                const uint32_t at = lanes + C::TM_O + blk * NR + r0 + g;
                uint32_t raw[16];
                tmem_ld16(at, raw);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) raw[i] = __float_as_uint(__uint_as_float(raw[i]) * row_by[r0 + g + i]);
                tmem_st16(at, raw);
              }
            tmem_st_wait();
          }
        }
        kv = words.get(t + 1, tile0 + kKeys);  // (asked for long before; used in the next turn)
        // weights, eight rows of a key side by side, into the buffer that the products of tile
        // t - 2 have read: the scores' commit came behind them
        const uint32_t weights = base + C::OFF_P + (t & 1) * C::P_BYTES + r0 / 8 * (kKeys * 16) + kt * 16;
#pragma unroll
        for (int r = 0; r < RPT; r += 8) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int y = r + 2 * i;
            const float w0 = ex2_approx(x[y]), w1 = ex2_approx(x[y + 1]);
            fma2(l[y], l[y + 1], w0, w1, mine_f.v_inv, mine_f.v_inv, l[y], l[y + 1]);
            w[i] = pack_f16x2(w0, w1);
            // (the offsets with the rounded weights, as the codes have them)
            fma2(ofs[y], ofs[y + 1], half_lo(w[i]), half_hi(w[i]), mine_f.v_ofs, mine_f.v_ofs, ofs[y], ofs[y + 1]);
          }
          st_shared_v4(weights + r / 8 * (kKeys * 16), w[0], w[1], w[2], w[3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        warp_arrive(bar(C::P_FULL + (t & 1)), lane);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");  // (none is left but where a wait ran out)

      // ---- epilogue: sums over the keys, then O
      {
        const float y = warp_sums<RPT>(l, lane), z = warp_sums<RPT>(ofs, lane);
        constexpr int GL = 32 / RPT;  // lanes that hold a row's sums
        if (lane % GL == 0) {
          red[(r0 + lane / GL) * 4 + w4] = y;
          red[(NR + r0 + lane / GL) * 4 + w4] = z;
        }
      }
      if (tiles > 0) wait(C::DRAIN, 0);
      const bool good = tiles > 0 && ok && *abort_flag == 0;
      named_barrier(nbar, 128);
      const bool whole = it.splits == 1;
      const long long first_part = static_cast<long long>(it.part - it.b) * p.T * p.H;  // (rows count from sequence 0)
      if (kt < rows_here) {
        const int r = r0 + kt, out = row_out[r];
        const float4 l4 = *reinterpret_cast<const float4*>(red + r * 4);
        const float4 o4 = *reinterpret_cast<const float4*>(red + (NR + r) * 4);
        const float ref = row_ref[r];
        float L = l4.x + l4.y + l4.z + l4.w;
        // (a row that saw no key has sums of 0; one whose scores are all NaN has NaN, and shows it)
        if (!own_live || !good) L = 0.f;
        row_add[r] = o4.x + o4.y + o4.z + o4.w;
        row_inv[r] = L == 0.f ? 0.f : (whole ? 1.f / L : 1.f);
        if (!whole) {
          p.part_m[first_part + out] = L == 0.f ? -INFINITY : ref;
          p.part_l[first_part + out] = L;
        } else if (p.lse) {
          p.lse[(static_cast<long long>(it.b) * p.H + out % p.H) * p.T + own_t] =
              L == 0.f ? -INFINITY : (ref + __log2f(L)) * 0.69314718055994531f;
        }
      }
      named_barrier(nbar, 128);
      // (of 64 features: sixteen in each quarter of the lanes)
      const int m = C::FB == 64 ? 16 * w4 + lane : kt, in8 = feature_at(m & 7);
      const bool holds = C::FB == 128 || lane < 16;
      const float unit = in8 & 1 ? 1048576.f : 16777216.f;  // (codes are 2^-24, odd features 2^-20)
#pragma unroll 1
      for (int blk = 0; blk < BLKS; ++blk) {
        const int f = blk * 128 + (m & ~7) + in8;
#pragma unroll 1
        for (int g = 0; g < rows_here; g += 16) {
          uint32_t raw[16];
          tmem_ld16(lanes + C::TM_O + blk * NR + r0 + g, raw);
          tmem_ld_wait();
          if (holds && f < (whole ? p.d : W)) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              if (g + i >= rows_here) break;
              const int r = r0 + g + i;
              const float a = row_inv[r];
              // (a row without keys: what lies there may be anything)
              const float o = a != 0.f ? fmaf(__uint_as_float(raw[i]), unit, row_add[r]) * a : 0.f;
              const long long row = row_out[r];
              if (whole) static_cast<__nv_bfloat16*>(p.out)[row * p.d + f] = __float2bfloat16_rn(o);
              else p.part_o[(first_part + row) * W + f] = o;
            }
          }
          __syncwarp();
        }
      }
      tc_fence_before();
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

template <class C>
cudaError_t launch_cfg(const RowsParams& p, cudaStream_t stream, LaunchInfo* info) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static bool attr_set[64] = {};
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    // (the softmax warps' registers come from those that a CTA is launched with)
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, rows_q4_many_kernel<C>);
    if (e != cudaSuccess) return e;
    if (attr.numRegs < C::REGS) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(rows_q4_many_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  const dim3 grid(static_cast<unsigned>(p.B * p.units * p.n_splits));
  e = launch_serialized(rows_q4_many_kernel<C>, grid, dim3(C::THREADS), C::SMEM, stream, p);
  if (info) {
    info->kernels = 1;
    info->grid = static_cast<int>(grid.x);
    info->block = C::THREADS;
    info->smem = C::SMEM;
  }
  return e;
}

// Calls f with the kernel's configuration for R rows per key head of d features.  Units of 32
// rows up to 32: they hold half the weights (8 x 24 heads of 128 features x 2,048 to 4,096
// keys, 32 rows: 49 us, 67 in units of 64).  Units of 64 from there on: each unpacks the
// tiles once for all of them (56 rows 68 us, in two units of 32 81; 252 rows 232 and 311).
// 16 or 32 rows to a softmax thread: four or two warpgroups.  64 features: 111.6 us (56 rows,
// 48 heads) with 16 and 112.5 with 32; 128: 92 and 68, where registers do not hold 16 warps'.
template <typename F>
void with_many(int d, int R, F&& f) {
  if (d <= 64) {
    f(ManyCfg<64, 64, 16, 2, 8>{});
  } else if (d <= 128) {
    if (R <= 32) f(ManyCfg<128, 32, 16, 2, 8>{});
    else f(ManyCfg<128, 64, 32, 2, 8>{});
  } else {
    if (R <= 32) f(ManyCfg<256, 32, 16, 3, 4>{});
    else f(ManyCfg<256, 64, 32, 3, 3>{});
  }
}

}  // namespace

RowsQ4Shape rows_q4_many_shape(int d, int R) {
  RowsQ4Shape s = {};
  with_many(d, R, [&](auto cfg) {
    using C = decltype(cfg);
    s.width = C::W;
    s.rows = C::NR;
    s.ctas = 1;
  });
  return s;
}

void rows_q4_many_ring(int slots, int tiles, int* loads, int* keys, int* values) {
  const RingItems items{slots, tiles};
  for (int x = 0; x < 2 * tiles; ++x, loads += 4) {
    const bool v = items.is_values(x);
    loads[0] = items.slot(x);
    loads[1] = v;
    loads[2] = items.tile(x);
    loads[3] = (v ? slots : 0) + items.slot(x);
  }
  SlotParity landed[2];
  for (int t = 0; t < tiles; ++t, keys += 3, values += 3) {
    keys[0] = items.keys(t);
    keys[1] = items.slot(keys[0]);
    keys[2] = landed[0].next(keys[1]);
    values[0] = items.values(t);
    values[1] = slots + items.slot(values[0]);
    values[2] = landed[1].next(items.slot(values[0]));
  }
}

cudaError_t launch_rows_q4_many(const RowsParams& p, cudaStream_t stream, LaunchInfo* info) {
  cudaError_t e = cudaSuccess;
  with_many(p.d, p.T * p.G, [&](auto cfg) { e = launch_cfg<decltype(cfg)>(p, stream, info); });
  return e;
}

}  // namespace mha

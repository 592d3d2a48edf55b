// Dense softmax attention over packed sequences with grouped heads, causal or
// full: the forward pass.
//
// What it computes, per sequence of Lq query and Lk key rows and query head h
// (key head h / G): row r sees its first n(r) keys, n(r) = Lk or, causal,
// clamp(r + 1 + Lk - Lq, 0, Lk);
//   lse(r) = log sum_{j < n(r)} exp(scale q_r . k_j)
//   out(r) = sum_{j < n(r)} exp(scale q_r . k_j - lse(r)) v_j
// and a row that sees nothing gives out = 0, lse = -inf.
//
// How (sm_100a).  A work item holds two 128-row query tiles ("slots") that
// share each K/V tile of 128 keys: neighbours in the list (row tile, head of
// the group) of one key head, so the two heads of an even group read the same
// rows and see the same keys, and with one head per key head the slots are
// neighbouring row tiles.  Per slot and key tile
//   S[128][128] = Q . K^T       (operands in shared memory)
//   O[128][D]  += P . V         (P in TMEM over its own S, V from shared memory)
// The tensor pipe alternates between the slots, so one slot's softmax runs
// under the other slot's products.  With at most two query tiles
// per SM an item is one of them: both slots have it, take its key tiles in turn,
// and their results are joined on the way out.  At D = 128 a product takes 596
// cycles with its A operand in TMEM and 861 with it in shared memory (measured:
// A's loads do not overlap the products), so 1457 per tile bound the rate; the
// TMEM of one SM is full (S and O of two slots), which keeps Q out of it in this
// form.
//
// One CTA per SM, 768 threads, item after item:
//   warp 0      K and V tiles (one ring of NST stages, K(j) then V(j))
//   warp 1      TMEM owner; one thread issues PV(j) and S(j+1) of slot 0, then of
//               slot 1, back to back, having waited for their tiles before
//   warp 2      zeroes what a sequence's last V tile holds past its keys (other
//               sequences' rows: their probabilities are 0, but 0 * inf is not)
//   warp 3      finds the work items, loads their Q tiles
//   warps 4-11, 12-19   softmax of slot 0, slot 1, 16 rows a warp (softmax_tile)
//   warps 20-23 epilogue: O / l, bf16 rows
// Measured on 15488 rows, 40 heads over 8, causal: 2.06-2.18 ms, 1130-1190 TFLOP/s
// (0.69-0.73 of the measured bf16 peak), about 1650 cycles a tile; called back to
// back, under the power limit, 2.39 ms.  (An earlier form with four softmax warps
// a slot, one row per thread: 2.51 ms single, where this one had 2.14.)  Part of
// the exponentials run on the FMA pipe (DENSE_POLY8 0 / 1 / 2 / 3 of 8: 745, 753,
// 725, 739 us on three full clips of 3000 to 9216 rows; the special-function unit
// alone does 16 a cycle).
// P is rounded to bf16 for the tensor core (half a step is at most 2^-8 of a
// value, and its error averages over the keys); sums, maxima and O stay fp32.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "dense_attn.cuh"
#include "dense_launch.h"
#include "vsa.h"
#include "vsa_device.cuh"

namespace vsa {
namespace dense {

using slim::mbar_wait;
using slim::warp_wait;

constexpr int kThreads = 768;
#ifndef DENSE_POLY8
#define DENSE_POLY8 2  // column pairs in eight whose exponential runs on the FMA pipe
#endif

// One slot of a work item.
struct Slot {
  int head;   // query head
  int row0;   // first row in q
  int rows;   // real rows (0: no such slot)
  int lim0;   // keys that tile row 0 sees (causal: row r sees lim0 + r, may be <= 0)
  int n;      // key tiles
  int last;   // keys that the last real row sees
};

struct Item {
  int n;  // key tiles; slot 0 has no fewer of them than slot 1
  int hk, kv0, kv_len;
  Slot slot0, slot1;
};
__device__ __forceinline__ const Slot& slot_of(const Item& x, int s) { return s ? x.slot1 : x.slot0; }

using Items = ItemRing<Item, 2>;

template <int D>
struct Layout {
  static constexpr int DH = D / 64;
  static constexpr uint32_t kTile = 128u * D * 2u;  // Q, K or V tile, bf16
  static constexpr int NST = D == 128 ? 5 : 10;     // K/V ring
  static constexpr uint32_t kQOff = 0;               // [2]
  static constexpr uint32_t kRingOff = kQOff + 2 * kTile;
  static constexpr uint32_t kMLOff = kRingOff + NST * kTile;  // [2][max, sum][128] f32
  static constexpr uint32_t kItemOff = kMLOff + 2048u;
  static constexpr uint32_t kBarOff = kItemOff + (uint32_t)sizeof(Items);
  static constexpr int kQFull = 0, kQEmpty = 2, kFull = 4, kEmpty = kFull + NST,
                       kPre = kEmpty + NST, kSFull = kPre + NST, kPFull = kSFull + 2,
                       kLFull = kPFull + 2, kOFull = kLFull + 2, kOEmpty = kOFull + 2,
                       kItFull = kOEmpty + 2, kItEmpty = kItFull + Items::kSlots, kTake = kItEmpty + Items::kSlots, kLoaded = kTake + 1, kNumBars = kLoaded + 1;
  static constexpr uint32_t kMiscOff = kBarOff + 8u * kNumBars;  // tmem address, abort flag
  static constexpr uint32_t kTakeOff = (kMiscOff + 16u + 15u) & ~15u;
  static constexpr uint32_t kAlloc = kTakeOff + 16u;
  static_assert(kAlloc <= 227u * 1024u, "shared memory");
};

// TMEM columns: S of slot s at 128 s (P in its first 64), O at 256 + D s.
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 256;

// Unit of a sequence: `slots` neighbours of the list u = row tile * G + head
// of the group, taken from the list's end (so slot 0 is the longer one and a
// list of odd length leaves its single slot to the shortest unit).
__device__ __forceinline__ Slot get_slot(const DenseParams& p, const int4& seq, int hk, int u) {
  Slot o;
  if (u < 0) {
    o.head = o.row0 = o.rows = o.lim0 = o.n = o.last = 0;
    return o;
  }
  const int tile = u / p.group;
  o.head = hk * p.group + (u - tile * p.group);
  o.row0 = seq.x + 128 * tile;
  o.rows = min(128, seq.y - 128 * tile);
  o.lim0 = p.causal ? seq.w - seq.y + 128 * tile + 1 : seq.w;
  o.last = p.causal ? max(0, o.lim0 + o.rows - 1) : seq.w;
  o.n = (o.last + 127) >> 7;
  return o;
}

__device__ __forceinline__ Item load_item(const DenseParams& p, const DenseSeqs& t, int w) {
  Item x;
  x.hk = w % p.Hkv;
  const Unit un = find_unit(t, w / p.Hkv);
  const int4 seq = t.seq[un.seq];
  x.kv0 = seq.z;
  x.kv_len = seq.w;
  const int u0 = ((seq.y + 127) >> 7) * p.group - 1 - p.slots * (t.units[un.seq] - 1 - un.rank);
  x.slot0 = get_slot(p, seq, x.hk, u0);
  x.n = x.slot0.n;
  if (p.slots == 2) {
    x.slot1 = get_slot(p, seq, x.hk, u0 - 1);
  } else {
    x.slot1 = x.slot0;
    x.slot0.n = (x.n + 1) >> 1;
    x.slot1.n = x.n >> 1;
  }
  return x;
}

// Row r of a slot, which sees no key.
template <int D>
__device__ __forceinline__ void unseen_row(const DenseParams& p, const Slot& sl, int r) {
  __nv_bfloat16* to = p.out + sl.head * p.out_st.h + (long long)(sl.row0 + r) * p.out_st.s;
  for (int e = 0; e < D; e += 8) *reinterpret_cast<uint4*>(to + e) = make_uint4(0u, 0u, 0u, 0u);
  if (p.lse) p.lse[sl.head * p.lse_seq + sl.row0 + r] = -INFINITY;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    dense_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ DenseParams p,
                     const __grid_constant__ DenseSeqs seqs) {
  using L = Layout<D>;
  constexpr int NST = L::NST;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {  // the tiles' swizzle needs it; there is no room to align by hand
    set_status(p.status, VSA_ERR_UNSUPPORTED);
    return;
  }
  float* ml = reinterpret_cast<float*>(smem + L::kMLOff);
  const bool turns = p.slots == 1;  // the slots take an item's key tiles in turn
  Items* items = reinterpret_cast<Items*>(smem + L::kItemOff);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);

  const int tid = threadIdx.x;
  const int warp = tid / 32, lane = tid % 32;

  // the first item takes a search in memory: before all else
  Item first = {};
  if (warp == 3) first = load_item(p, seqs, blockIdx.x);

  if (warp == 0) {
    for (int i = lane; i < L::kNumBars; i += 32) {
      // a TMA transaction, a commit or one thread's arrival, except where warps arrive
      const uint32_t count = (i >= L::kPFull && i < L::kOFull)    ? 8u  // a slot's softmax
                             : (i >= L::kOEmpty && i < L::kItFull) ? 4u  // the epilogue
                             : (i >= L::kItEmpty && i < L::kTake)  ? kThreads / 32 - 1u
                                                                   : 1u;
      mbar_init(bars + i, count);
    }
    if (lane == 0) {
      abort_flag[0] = 0;
      abort_flag[1] = p.item_us;
    }
    mbar_fence_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  auto next = [&](uint32_t& w, Item& x) {
    return get_item(items, bars + L::kItFull, bars + L::kItEmpty, w, x, lane, abort_flag, p.status);
  };

  if (warp == 0) {
    // ===================== K and V tiles =====================
    const uint64_t pol = l2_policy_evict_last();
    uint32_t g = 0, n_got = 0;
    bool ok = true;
    Item x;
    while (ok && next(n_got, x)) {
      if (lane == 0) {
        for (int j = 0; ok && j < 2 * x.n; ++j, ++g) {
          const int st = (int)(g % NST);
          const uint32_t u = g / NST;
          if (u >= 1) ok = mbar_wait(bars + L::kEmpty + st, (u - 1) & 1, abort_flag, p.status);
          if (!ok) break;
          const bool is_v = j & 1;
          const int key = 128 * (j >> 1);
          // a V tile with rows past the sequence goes through warp 2 first
          uint64_t* full = bars + (is_v && x.kv_len - key < 128 ? L::kPre : L::kFull) + st;
          uint8_t* dst = smem + L::kRingOff + st * L::kTile;
          mbar_arrive_expect_tx(full, L::kTile);
#pragma unroll
          for (int dh = 0; dh < L::DH; ++dh)
            load_rows(dst + dh * 16384, is_v ? &tm_v : &tm_k, is_v ? p.v_ax : p.k_ax, full, dh * 64, x.kv0 + key,
                      x.hk, 0, pol);
        }
        mbar_arrive(bars + L::kLoaded);
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
    }
    __syncwarp();
  } else if (warp == 3) {
    // ===================== work items and their Q tiles =====================
    const uint64_t pol = l2_policy_evict_first();
    uint32_t n = 0, cs0 = 0, cs1 = 0;  // items; Q tiles of the slots
    bool ok = true;
    Item x = first;
    Takeover take{bars + L::kTake, reinterpret_cast<uint4*>(smem + L::kTakeOff), 0};
    for (int it = blockIdx.x; ok && it >= 0; it = ok ? take.answer(abort_flag, p.status) : -1) {
      if (it != (int)blockIdx.x) x = load_item(p, seqs, it);
      if (x.n == 0) {
        // nothing to multiply: not handed on (the products look one item ahead, and
        // must not wait for one past those that the others have taken)
#pragma unroll 1
        for (int s = 0; s < p.slots; ++s) {
          const Slot& sl = slot_of(x, s);
          for (int r = lane; r < sl.rows; r += 32) unseen_row<D>(p, sl, r);
        }
        take.ask(lane);
        continue;
      }
      ok = put_item(items, bars + L::kItFull, bars + L::kItEmpty, n, x, lane, abort_flag, p.status);
#pragma unroll 1
      for (int s = 0; ok && s < 2; ++s) {
        const Slot& sl = slot_of(x, s);
        if (sl.n == 0) continue;
        const uint32_t cs = s ? cs1 : cs0;
        if (cs >= 1) ok = warp_wait(bars + L::kQEmpty + s, (cs - 1) & 1, abort_flag, p.status);
        if (!ok) break;
        cs0 += s ^ 1;
        cs1 += s;
        if (lane == 0) {
          mbar_arrive_expect_tx(bars + L::kQFull + s, L::kTile);
#pragma unroll
          for (int dh = 0; dh < L::DH; ++dh)
            load_rows(smem + L::kQOff + s * L::kTile + dh * 16384, &tm_q, p.q_ax, bars + L::kQFull + s, dh * 64,
                      sl.row0, sl.head, 0, pol);
        }
        __syncwarp();
      }
      // ask for more when this item's last tiles are on their way, not earlier: what
      // a CTA holds no other can take
      ok = ok && warp_wait(bars + L::kLoaded, n++ & 1, abort_flag, p.status);
      if (ok) take.ask(lane);
    }
    x.n = -1;
    if (ok) put_item(items, bars + L::kItFull, bars + L::kItEmpty, n, x, lane, abort_flag, p.status);
  } else if (warp == 2) {
    // ===================== zero V rows past a sequence's keys =====================
    uint32_t g = 0, pre = 0, n_got = 0;  // ring tiles so far; phase bit per stage
    Item x;
    while (next(n_got, x)) {
      g += 2 * x.n;
      const int len = x.kv_len - 128 * (x.n - 1);  // keys from the last loaded tile on
      if (len >= 128) continue;
      const int st = (int)((g - 1) % NST);
      if (!warp_wait(bars + L::kPre + st, (pre >> st) & 1, abort_flag, p.status)) break;
      pre ^= 1u << st;
      // products stop at the next multiple of 16 keys
      zero_rows<128>(smem + L::kRingOff + st * L::kTile, L::DH, len, (len + 15) & ~15, lane);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + L::kFull + st);
    }
  } else if (warp == 1) {
    // ===================== MMA issue: one thread =====================
    if (elect_one()) {
      uint32_t q0 = 0, q1 = 0;  // items of the slots whose first S was issued
      uint32_t d0 = 0, d1 = 0;  // items of the slots whose products are issued
      uint32_t p0 = 0, p1 = 0;  // key tiles of the slots whose P has been consumed
      uint32_t g = 0, n_got = 0;
      bool ok = true;
      auto wait = [&](int bar, uint32_t ph) {
        if (!mbar_wait(bars + bar, ph & 1, abort_flag, p.status)) ok = false;
      };
      auto tile = [&](uint32_t at) { return sbase + L::kRingOff + (at % NST) * L::kTile; };
      auto wait_stage = [&](uint32_t at) { wait(L::kFull + (int)(at % NST), at / NST); };
      // which key tile is the j-th of slot s; whether slot s is the last to read it
      auto key_tile = [&](int s, int j) { return turns ? 2 * j + s : j; };
      auto last_reader = [&](const Item& x, int s, int j) { return turns || s == 1 || j >= x.slot1.n; };
      // what S(j) of slot s waits for, and S(j); the item's ring tiles start at gx
      auto before_s = [&](int s, int j, uint32_t gx) {
        if (j == 0) {
          wait(L::kQFull + s, s ? q1 : q0);
          q0 += s ^ 1;
          q1 += s;
        }
        wait_stage(gx + 2 * key_tile(s, j));
      };
      auto do_s = [&](const Item& x, int s, int j, uint32_t gx) {
        const uint32_t at = gx + 2 * key_tile(s, j);
        issue_s<D>(tmem_base + 128u * s, sbase + L::kQOff + s * L::kTile, tile(at));
        umma_commit(bars + L::kSFull + s);
        if (last_reader(x, s, j)) umma_commit(bars + L::kEmpty + (int)(at % NST));
        if (j == slot_of(x, s).n - 1) umma_commit(bars + L::kQEmpty + s);
      };
      auto next_one = [&](Item& x) {
        return get_item_one(items, bars + L::kItFull, bars + L::kItEmpty, n_got, x, abort_flag, p.status);
      };
      Item x, y;
      bool have = next_one(x);
#pragma unroll 1
      for (int s = 0; ok && have && s < 2; ++s) {
        if (slot_of(x, s).n == 0) continue;
        before_s(s, 0, 0);
        if (!ok) break;
        tc_fence_after_sync();
        do_s(x, s, 0, 0);
      }
      while (ok && have) {
        bool more = false;
        const uint32_t g_next = g + 2 * x.n;
        const int n0 = x.slot0.n, n1 = x.slot1.n;
#pragma unroll 1
        for (int i = 0; ok && i < 2 * n0; ++i) {
          const int s = i & 1, j = i >> 1, ns = s ? n1 : n0;
          if (j >= ns) {
            // slot 1 is through; its next item begins when slot 0 is, too
            if (j == n0 - 1 && more && y.slot1.n > 0) {
              before_s(1, 0, g_next);
              if (!ok) break;
              tc_fence_after_sync();
              do_s(y, 1, 0, g_next);
            }
            continue;
          }
          // PV(j), then the next S: within an item what S will need first, so that it
          // follows at once (the next item's Q may still be on its way)
          const bool last = j + 1 == ns;
          const uint32_t gv = g + 2 * key_tile(s, j) + 1;
          wait_stage(gv);
          // (the item's tiles are here or on their way, so that the next one was asked for)
          if (s == 0 && last && ok) more = next_one(y);
          if (!last) before_s(s, j + 1, g);
          // the epilogue has emptied this slot's O
          const uint32_t done = s ? d1 : d0;
          if (j == 0 && done >= 1) wait(L::kOEmpty + s, done - 1);
          wait(L::kPFull + s, s ? p1 : p0);
          p0 += s ^ 1;
          p1 += s;
          if (!ok) break;
          tc_fence_after_sync();
          const int keys = slot_of(x, s).last - 128 * key_tile(s, j);
          issue_pv<D>(tmem_base + kTmemO + D * s, tmem_base + 128u * s, tile(gv),
                      keys >= 128 ? 8 : (keys + 15) >> 4, j > 0);
          if (last_reader(x, s, j)) umma_commit(bars + L::kEmpty + (int)(gv % NST));
          if (last) {
            umma_commit(bars + L::kOFull + s);
            d0 += s ^ 1;
            d1 += s;
          }
          if (!last) {
            do_s(x, s, j + 1, g);
          } else if (j == n0 - 1 && more && slot_of(y, s).n > 0) {
            before_s(s, 0, g_next);
            if (!ok) break;
            tc_fence_after_sync();
            do_s(y, s, 0, g_next);
          }
        }
        g = g_next;
        x = y;
        have = more;
      }
    }
    __syncwarp();
  } else if (warp < 20) {
    // ===================== softmax: 16 query rows a warp =====================
    const int s = (warp - 4) >> 3, upper = (warp - 4) >> 2 & 1;
    const int first_row = 32 * (warp & 3) + 16 * upper;  // TMEM lane = query row
    const uint32_t t_s = tmem_base + ((uint32_t)first_row << 16) + 128u * s;
    const uint32_t t_o = tmem_base + ((uint32_t)first_row << 16) + kTmemO + D * s;
    uint32_t g = 0, n = 0, n_got = 0;
    bool ok = true;
    Item x;
    while (ok && next(n_got, x)) {
      const Slot sl = slot_of(x, s);
      if (sl.n == 0) continue;
      float m[2] = {-INFINITY, -INFINITY};
      uint64_t l2[2] = {0, 0};
      for (int j = 0; j < sl.n; ++j, ++g) {
        // columns of the tile that rows see: one more per row where causal
        const int key = 128 * (turns ? 2 * j + s : j);
        int rem[2], whole = x.kv_len - key, none = whole;
        rem[0] = rem[1] = whole;
        if (p.causal) {
          const int r0 = sl.lim0 + first_row - key;
          rem[0] = min(whole, r0 + lane / 4);
          rem[1] = min(whole, r0 + lane / 4 + 8);
          none = min(whole, r0 + 15);
          whole = min(whole, r0);
        }
        if (!warp_wait(bars + L::kSFull + s, g & 1, abort_flag, p.status)) { ok = false; break; }
        tc_fence_after_sync();
        softmax_tile<D, DENSE_POLY8, 2>(t_s, t_o, p.scale_log2, rem, whole, none, j == 0, lane, m, l2);
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + L::kPFull + s);
      }
      if (!ok) break;
      // hand max and sum to the epilogue, once it has taken the previous item's
      if (n >= 1 && !warp_wait(bars + L::kOEmpty + s, (n - 1) & 1, abort_flag, p.status)) { ok = false; break; }
      ++n;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const float l = quad_sum(l2[b]);
        if ((lane & 3) == 0) {
          ml[s * 256 + first_row + lane / 4 + 8 * b] = m[b];
          ml[s * 256 + 128 + first_row + lane / 4 + 8 * b] = l;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + L::kLFull + s);
    }
  } else {
    // ===================== epilogue: one thread per query row =====================
    const int row = 32 * (warp & 3) + lane;
    const uint32_t t_lane = tmem_base + (uint32_t(32 * (warp & 3)) << 16) + kTmemO;
    uint32_t cs0 = 0, cs1 = 0, n_got = 0;
    bool ok = true;
    Item x;
    while (ok && next(n_got, x)) {
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {
        // the shorter slot (1) ends first where the two differ
        const int s = x.slot1.n < x.slot0.n ? 1 - k : k;
        const Slot sl = slot_of(x, s);
        if (sl.rows == 0) continue;
        const bool real = row < sl.rows;
        if (sl.n == 0) {
          if (real && !turns) unseen_row<D>(p, sl, row);
          continue;
        }
        const uint32_t ph = (s ? cs1 : cs0) & 1;
        cs0 += s ^ 1;
        cs1 += s;
        if (!warp_wait(bars + L::kLFull + s, ph, abort_flag, p.status) ||
            !warp_wait(bars + L::kOFull + s, ph, abort_flag, p.status)) { ok = false; break; }
        // slots that took turns are written together
        const bool both = turns && x.slot1.n > 0;
        if (both && k == 0) continue;
        tc_fence_after_sync();
        const int s0 = both ? 0 : s;
        float top = ml[s0 * 256 + row], sum = ml[s0 * 256 + 128 + row], w0 = 1.f, w1 = 0.f;
        if (both) {
          const float m0 = top, m1 = ml[256 + row], l1 = ml[384 + row];
          top = fmaxf(m0, m1);
          const float ref = top == -INFINITY ? 0.f : top;
          w0 = fast_exp2(m0 - ref);
          w1 = fast_exp2(m1 - ref);
          sum = sum * w0 + l1 * w1;
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        w0 *= inv;
        w1 *= inv;
        if (p.lse && real)
          p.lse[sl.head * p.lse_seq + sl.row0 + row] =
              sum == 0.f ? -INFINITY : (top + __log2f(sum)) * 0.69314718055994531f;
        __nv_bfloat16* orow = p.out + sl.head * p.out_st.h + (long long)(sl.row0 + row) * p.out_st.s;
#pragma unroll 1
        for (int q0 = 0; q0 < D; q0 += 16) {
          uint32_t ov[16], o1[16];
          VSA_TMEM_LD16(t_lane + D * s0 + q0, ov, 0);
          if (both) VSA_TMEM_LD16(t_lane + D + q0, o1, 0);
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
          if (q0 + 16 == D) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(bars + L::kOEmpty + s0);
              if (both) mbar_arrive(bars + L::kOEmpty + 1);
            }
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float f = __uint_as_float(ov[e]) * w0;
            if (both) f = fmaf(__uint_as_float(o1[e]), w1, f);
            ov[e] = __float_as_uint(f);
          }
          if (real) {
#pragma unroll
            for (int e = 0; e < 16; e += 8)
              *reinterpret_cast<uint4*>(orow + q0 + e) = make_uint4(
                  pack_bf16x2(__uint_as_float(ov[e]), __uint_as_float(ov[e + 1])),
                  pack_bf16x2(__uint_as_float(ov[e + 2]), __uint_as_float(ov[e + 3])),
                  pack_bf16x2(__uint_as_float(ov[e + 4]), __uint_as_float(ov[e + 5])),
                  pack_bf16x2(__uint_as_float(ov[e + 6]), __uint_as_float(ov[e + 7])));
          }
        }
      }
    }
  }

  settle_after_abort(abort_flag);
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

}  // namespace dense

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int device_sm_count() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

int KernelReady::check(const void* kern, int smem) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return VSA_ERR_CUDA;
  const unsigned long long bit = 1ull << dev;
  if (done.load(std::memory_order_acquire) & bit) return VSA_OK;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return VSA_ERR_CUDA;
  done.fetch_or(bit, std::memory_order_release);
  return VSA_OK;
}

int DenseBatch::chunk(int i0, int4* seqs) const {
  const int m = n - i0 < kDenseMaxSeqs ? n - i0 : kDenseMaxSeqs;
  for (int i = 0; i < m; ++i)
    seqs[i] = make_int4(cu_q[i0 + i], cu_q[i0 + i + 1] - cu_q[i0 + i], cu_kv[i0 + i],
                        cu_kv[i0 + i + 1] - cu_kv[i0 + i]);
  return m;
}

int item_microseconds(const DenseBatch& b, bool over_rows, int group) {
  long long tiles = 0;
  for (int i = 0; i < b.n; ++i) {
    const int32_t* cu = over_rows ? b.cu_q : b.cu_kv;
    tiles = std::max(tiles, (cu[i + 1] - cu[i] + 127LL) / 128 * group);
  }
  return (int)std::min(20 * tiles, 1000000000LL);
}

void fill_dense_seqs(DenseSeqs* t, const int4* seqs, const int* units, const int* flat_cost, int n) {
  int order[kDenseMaxSeqs];
  int m = 0;
  for (int i = 0; i < n; ++i)
    if (units[i] > 0) order[m++] = i;
  std::stable_sort(order, order + m, [&](int a, int b) {
    if ((flat_cost[a] > 0) != (flat_cost[b] > 0)) return flat_cost[a] > 0;
    return flat_cost[a] > 0 ? flat_cost[a] > flat_cost[b] : units[a] > units[b];
  });
  t->n = m;
  t->n_flat = 0;
  int at = 0;
  for (int r = 0; r < m; ++r) {
    t->seq[r] = seqs[order[r]];
    t->units[r] = units[order[r]];
    if (flat_cost[order[r]] > 0) {
      t->first[r] = at;
      at += t->units[r];
      t->n_flat = r + 1;
    }
  }
  t->first[t->n_flat] = at;
  for (int k = t->n_flat + 1; k <= m; ++k) {
    t->first[k] = at;
    at += (k - t->n_flat) * (t->units[k - 1] - (k < m ? t->units[k] : 0));
  }
  t->n_units = at;
}

template <int D>
static int launch_dense_fwd_t(DenseParams p, const DenseSeqs& seqs, const CUtensorMap& mq,
                              const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t stream) {
  using L = dense::Layout<D>;
  auto kern = dense::dense_fwd_kernel<D>;
  static KernelReady ready;
  const int rc = ready.check(reinterpret_cast<const void*>(kern), (int)L::kAlloc);
  if (rc != VSA_OK) return rc;
  const int grid = seqs.n_units * p.Hkv;
  if (grid == 0) return VSA_OK;
  kern<<<(unsigned)grid, dense::kThreads, L::kAlloc, stream>>>(mq, mk, mv, p, seqs);
  return cudaGetLastError() == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
}

int launch_dense_fwd(const DenseParams& p_in, const DenseTensors& t, const DenseBatch& b, int D,
                     cudaStream_t stream) {
  DenseParams p = p_in;
  CUtensorMap mq, mk, mv;
  if (!make_view_map_rows(&mq, &p.q_ax, t.q, D, t.q_seq, p.Hq, 1, t.q_st, 128)) return VSA_ERR_CUDA;
  // without keys no tile is loaded; the maps only have to be valid
  const bool keys = t.kv_seq > 0;
  if (!make_view_map_rows(&mk, &p.k_ax, keys ? t.k : t.q, D, keys ? t.kv_seq : t.q_seq,
                          keys ? p.Hkv : p.Hq, 1, keys ? t.k_st : t.q_st, 128) ||
      !make_view_map_rows(&mv, &p.v_ax, keys ? t.v : t.q, D, keys ? t.kv_seq : t.q_seq,
                          keys ? p.Hkv : p.Hq, 1, keys ? t.v_st : t.q_st, 128))
    return VSA_ERR_CUDA;
  p.item_us = item_microseconds(b, false, 1);
  for (int i0 = 0; i0 < b.n; i0 += kDenseMaxSeqs) {
    int4 seqs[kDenseMaxSeqs];
    int units[kDenseMaxSeqs], flat[kDenseMaxSeqs];
    const int n = b.chunk(i0, seqs);
    long long slots = 0;
    for (int i = 0; i < n; ++i) slots += (seqs[i].y + 127LL) / 128 * p.Hq;
    if (slots >= (1 << 30)) return VSA_ERR_UNSUPPORTED;  // 32-bit item index
    // Two row tiles per item halve the K/V reads; up to two tiles per SM, one
    // tile per item whose key tiles the slots share ends sooner (rows x heads, us
    // with pairs and with single tiles: 1000 x 20: 28.7, 20.5; 3000 x 12: 59.4,
    // 46.1; above it they tie: 1000 x 40: 30.7, 28.7-30.7; 2000 x 40: 61.4, 61.4).
    p.slots = slots > 2 * device_sm_count() ? 2 : 1;
    for (int i = 0; i < n; ++i) {
      units[i] = ((seqs[i].y + 127) / 128 * p.group + p.slots - 1) / p.slots;
      // behind cached keys the first rows, too, have many to see
      flat[i] = !p.causal || seqs[i].w > seqs[i].y ? seqs[i].w : 0;
    }
    DenseSeqs table;
    fill_dense_seqs(&table, seqs, units, flat, n);
    const int rc = D == 128 ? launch_dense_fwd_t<128>(p, table, mq, mk, mv, stream)
                            : launch_dense_fwd_t<64>(p, table, mq, mk, mv, stream);
    if (rc != VSA_OK) return rc;
  }
  return VSA_OK;
}

}  // namespace vsa

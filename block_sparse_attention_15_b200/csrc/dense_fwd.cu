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
// under the other slot's products: at D = 128 a tile costs 1024 tensor cycles
// and 1024 cycles of the exponential unit (16 per cycle), so part of the
// exponentials run on the FMA pipe (exp2_fma2).
//
// Persistent grid, one CTA per SM, 512 threads, four warpgroups:
//   warp 0      K and V tiles (one ring of NST stages, K(j) then V(j))
//   warp 1      TMEM owner; issues PV(j) and S(j+1) of slot 0, then of slot 1
//   warp 2      zeroes what a sequence's last V tile holds past its keys (other
//               sequences' rows: their probabilities are 0, but 0 * inf is not)
//   warp 3      Q tiles
//   warps 4-7, 8-11   softmax of slot 0, slot 1: one thread per query row, 128
//               columns in registers.  The reference max moves only when a
//               tile's max exceeds it by more than kRefresh log2 units; the
//               thread then rescales its O row itself (S(j) complete implies
//               PV(j-1) complete: one thread issued both, in order)
//   warps 12-15 epilogue: O / l, bf16 rows
// P is rounded to bf16 for the tensor core (half a step is 2^-9 of a value,
// and its error averages over the keys); sums, maxima and O stay fp32.
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

constexpr int kThreads = 512;
constexpr uint32_t kRegsProducer = 80, kRegsSoftmax = 184, kRegsEpilogue = 64;
constexpr uint32_t kLaunchRegs = 128;  // 512 x 128 = 65536
static_assert(128u * (kRegsProducer + 2u * kRegsSoftmax + kRegsEpilogue) <= 512u * kLaunchRegs,
              "register split exceeds the launch's registers");
// Largest excess (log2 units) of a logit over its row's reference max that is
// exponentiated without moving the reference: probabilities stay below 2^8.
constexpr float kRefresh = 8.f;
#ifndef DENSE_POLY8
#define DENSE_POLY8 2  // column pairs in eight whose exponential runs on the FMA pipe
#endif

template <int D>
struct Layout {
  static constexpr int DH = D / 64;
  static constexpr uint32_t kTile = 128u * D * 2u;  // Q, K or V tile, bf16
  static constexpr int NST = D == 128 ? 5 : 8;      // K/V ring
  static constexpr uint32_t kQOff = 0;               // [2]
  static constexpr uint32_t kRingOff = kQOff + 2 * kTile;
  static constexpr uint32_t kInvLOff = kRingOff + NST * kTile;  // [2][128] f32
  static constexpr uint32_t kBarOff = kInvLOff + 2u * 128u * 4u;
  static constexpr int kQFull = 0, kQEmpty = 2, kFull = 4, kEmpty = kFull + NST,
                       kPre = kEmpty + NST, kSFull = kPre + NST, kPFull = kSFull + 2,
                       kOFull = kPFull + 2, kOEmpty = kOFull + 2, kLFull = kOEmpty + 2,
                       kNumBars = kLFull + 2;
  static constexpr uint32_t kMiscOff = kBarOff + 8u * kNumBars;  // tmem address, abort flag
  static constexpr uint32_t kBytes = kMiscOff + 16u;
  static constexpr uint32_t kAlloc = kBytes + 1024u;
  static_assert(kAlloc <= 227u * 1024u, "shared memory");
};

// TMEM columns: S of slot s at 128 s (P in its first 64), O at 256 + D s.
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 256;

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
  int hk;
  int q0, q_len, kv0, kv_len;
  int u0;      // slot 0's place in the sequence's list of (row tile, head); slot 1's is u0 - 1
  int n0, n1;  // key tiles of the slots, n0 >= n1
};

__device__ __forceinline__ Slot get_slot(const DenseParams& p, const Item& x, int s) {
  Slot o;
  const int u = x.u0 - s;
  if (s >= p.slots || u < 0) {
    o.head = o.row0 = o.rows = o.lim0 = o.n = o.last = 0;
    return o;
  }
  const int tile = u / p.group;
  o.head = x.hk * p.group + (u - tile * p.group);
  o.row0 = x.q0 + 128 * tile;
  o.rows = min(128, x.q_len - 128 * tile);
  o.lim0 = p.causal ? x.kv_len - x.q_len + 128 * tile + 1 : x.kv_len;
  o.last = p.causal ? max(0, o.lim0 + o.rows - 1) : x.kv_len;
  o.n = (o.last + 127) >> 7;
  return o;
}

// Unit of a sequence: `slots` neighbours of the list u = row tile * G + head
// of the group, taken from the list's end (so slot 0 is the longer one and a
// list of odd length leaves its single slot to the shortest unit).
__device__ __forceinline__ Item load_item(const DenseParams& p, const DenseSeqs& t, int w) {
  Item x;
  x.hk = w % p.Hkv;
  const Unit un = find_unit(t, w / p.Hkv);
  const int4 q = t.seq[un.seq];
  x.q0 = q.x;
  x.q_len = q.y;
  x.kv0 = q.z;
  x.kv_len = q.w;
  x.u0 = ((q.y + 127) >> 7) * p.group - 1 - p.slots * (t.units[un.seq] - 1 - un.rank);
  x.n0 = get_slot(p, x, 0).n;
  x.n1 = get_slot(p, x, 1).n;
  return x;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    dense_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ DenseParams p,
                     const __grid_constant__ DenseSeqs seqs) {
  using L = Layout<D>;
  constexpr int NST = L::NST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  float* inv_l = reinterpret_cast<float*>(smem + L::kInvLOff);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);

  const int tid = threadIdx.x;
  const int warp = tid / 32, lane = tid % 32;
  const int cta = blockIdx.x, grid = gridDim.x;

  if (warp == 0) {
    for (int i = lane; i < L::kNumBars; i += 32) {
      // a TMA transaction, a commit or one thread's arrival, except where the
      // four warps of a softmax or epilogue group arrive
      const bool four = (i >= L::kPFull && i < L::kPFull + 2) || (i >= L::kOEmpty && i < L::kNumBars);
      mbar_init(bars + i, four ? 4u : 1u);
    }
    if (lane == 0) *abort_flag = 0;
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

  if (warp < 4) {
    regs_dec<kRegsProducer>();
    if (warp == 0) {
      // ===================== K and V tiles =====================
      if (lane == 0) {
        const uint64_t pol = l2_policy_evict_last();
        uint32_t g = 0;  // ring tiles so far
        bool ok = true;
        for (int w = 0, it; ok && (it = wave_item(w, cta, grid), w * grid < p.n_work); ++w) {
          if (it >= p.n_work) continue;
          const Item x = load_item(p, seqs, it);
          for (int j = 0; ok && j < 2 * x.n0; ++j, ++g) {
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
              load_rows(dst + dh * 16384, is_v ? &tm_v : &tm_k, is_v ? p.v_ax : p.k_ax, full,
                        dh * 64, x.kv0 + key, x.hk, 0, pol);
          }
        }
        // every stage's release lands before exit
        for (uint32_t t = (g > (uint32_t)NST ? g - NST : 0u); ok && t < g; ++t)
          ok = mbar_wait(bars + L::kEmpty + (int)(t % NST), (t / NST) & 1, abort_flag, p.status);
      }
      __syncwarp();
    } else if (warp == 3) {
      // ===================== Q tiles =====================
      if (lane == 0) {
        const uint64_t pol = l2_policy_evict_first();
        uint32_t cs[2] = {0, 0};
        bool ok = true;
        for (int w = 0, it; ok && (it = wave_item(w, cta, grid), w * grid < p.n_work); ++w) {
          if (it >= p.n_work) continue;
          const Item x = load_item(p, seqs, it);
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (!ok || (s ? x.n1 : x.n0) == 0) continue;
            const Slot sl = get_slot(p, x, s);
            if (cs[s] >= 1) ok = mbar_wait(bars + L::kQEmpty + s, (cs[s] - 1) & 1, abort_flag, p.status);
            if (!ok) continue;
            ++cs[s];
            mbar_arrive_expect_tx(bars + L::kQFull + s, L::kTile);
#pragma unroll
            for (int dh = 0; dh < L::DH; ++dh)
              load_rows(smem + L::kQOff + s * L::kTile + dh * 16384, &tm_q, p.q_ax,
                        bars + L::kQFull + s, dh * 64, sl.row0, sl.head, 0, pol);
          }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
          if (ok && cs[s]) ok = mbar_wait(bars + L::kQEmpty + s, (cs[s] - 1) & 1, abort_flag, p.status);
      }
      __syncwarp();
    } else if (warp == 2) {
      // ===================== zero V rows past a sequence's keys =====================
      uint32_t g = 0, pre = 0;  // ring tiles so far; phase bit per stage
      bool ok = true;
      for (int w = 0, it; ok && (it = wave_item(w, cta, grid), w * grid < p.n_work); ++w) {
        if (it >= p.n_work) continue;
        const Item x = load_item(p, seqs, it);
        if (x.n0 == 0) continue;
        g += 2 * x.n0;
        const int len = x.kv_len - 128 * (x.n0 - 1);  // keys from the last loaded tile on
        if (len >= 128) continue;
        const int st = (int)((g - 1) % NST);
        if (!warp_wait(bars + L::kPre + st, (pre >> st) & 1, abort_flag, p.status)) { ok = false; break; }
        pre ^= 1u << st;
        // products stop at the next multiple of 16 keys
        zero_rows<128>(smem + L::kRingOff + st * L::kTile, L::DH, len, (len + 15) & ~15, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + L::kFull + st);
      }
    } else {
      // ===================== MMA issue =====================
      uint32_t cs[2] = {0, 0};  // items of the slot that have started
      uint32_t gs[2] = {0, 0};  // key tiles of the slot whose P has been consumed
      uint32_t g = 0;            // ring tiles before the current item
      bool ok = true;
      // S(j) of slot s of item x, whose ring tiles start at g_item
      auto do_s = [&](const Item& x, int s, int j, uint32_t g_item) {
        const uint32_t gk = g_item + 2 * j;
        const int st = (int)(gk % NST);
        if (j == 0) {
          if (!warp_wait(bars + L::kQFull + s, cs[s] & 1, abort_flag, p.status)) { ok = false; return; }
          ++cs[s];
        }
        if (!warp_wait(bars + L::kFull + st, (gk / NST) & 1, abort_flag, p.status)) { ok = false; return; }
        tc_fence_after_sync();
        if (elect_one()) {
          issue_s<D>(tmem_base + 128u * s, sbase + L::kQOff + s * L::kTile, sbase + L::kRingOff + st * L::kTile);
          umma_commit(bars + L::kSFull + s);
          if (s == 1 || j >= x.n1) umma_commit(bars + L::kEmpty + st);
          if (j == (s ? x.n1 : x.n0) - 1) umma_commit(bars + L::kQEmpty + s);
        }
        __syncwarp();
      };
      // item iteration with one item of look-ahead
      int w = 0;
      auto next_item = [&](Item& x) -> bool {  // the next item with key tiles
        for (; w * grid < p.n_work; ++w) {
          const int it = wave_item(w, cta, grid);
          if (it >= p.n_work) continue;
          x = load_item(p, seqs, it);
          if (x.n0 > 0) { ++w; return true; }
        }
        return false;
      };
      Item x, y;
      bool have = next_item(x);
      if (have) {
        do_s(x, 0, 0, g);
        if (ok && x.n1 > 0) do_s(x, 1, 0, g);
      }
      while (ok && have) {
        const bool more = next_item(y);
        const uint32_t g_next = g + 2 * x.n0;
        const int last[2] = {get_slot(p, x, 0).last, get_slot(p, x, 1).last};
        for (int j = 0; ok && j < x.n0; ++j) {
          const uint32_t gv = g + 2 * j + 1;
          const int st = (int)(gv % NST);
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (!ok || j >= (s ? x.n1 : x.n0)) continue;
            // the epilogue has emptied this slot's O
            if (j == 0 && cs[s] >= 2 &&
                !warp_wait(bars + L::kOEmpty + s, (cs[s] - 2) & 1, abort_flag, p.status)) { ok = false; continue; }
            if (!warp_wait(bars + L::kFull + st, (gv / NST) & 1, abort_flag, p.status)) { ok = false; continue; }
            if (!warp_wait(bars + L::kPFull + s, gs[s] & 1, abort_flag, p.status)) { ok = false; continue; }
            ++gs[s];
            tc_fence_after_sync();
            if (elect_one()) {
              const int keys = last[s] - 128 * j;
              issue_pv<D>(tmem_base + kTmemO + D * s, tmem_base + 128u * s,
                          sbase + L::kRingOff + st * L::kTile, keys >= 128 ? 8 : (keys + 15) >> 4, j > 0);
              if (s == 1 || j >= x.n1) umma_commit(bars + L::kEmpty + st);
              if (j == (s ? x.n1 : x.n0) - 1) umma_commit(bars + L::kOFull + s);
            }
            __syncwarp();
            if (j + 1 < (s ? x.n1 : x.n0)) do_s(x, s, j + 1, g);
            else if (s == 0 && more) do_s(y, 0, 0, g_next);
          }
        }
        if (ok && more && y.n1 > 0) do_s(y, 1, 0, g_next);
        g = g_next;
        x = y;
        have = more;
      }
    }
  } else if (warp < 12) {
    regs_inc<kRegsSoftmax>();
    // ===================== softmax: one thread per query row =====================
    const int s = (warp - 4) >> 2;
    const int wq = warp & 3;
    const int row = wq * 32 + lane;  // TMEM lane = query row
    const uint32_t t_s = tmem_base + (uint32_t(wq * 32) << 16) + 128u * s;
    const uint32_t t_o = tmem_base + (uint32_t(wq * 32) << 16) + kTmemO + D * s;
    const float c = p.scale_log2;
    const uint64_t cc = pk2(c, c);
    uint32_t g = 0, n = 0;
    bool ok = true;
    for (int w = 0, it; ok && (it = wave_item(w, cta, grid), w * grid < p.n_work); ++w) {
      if (it >= p.n_work) continue;
      const Item x = load_item(p, seqs, it);
      const Slot sl = get_slot(p, x, s);
      if (sl.n == 0) continue;
      const int limit = p.causal ? min(sl.lim0 + row, x.kv_len) : x.kv_len;  // keys this row sees
      float m = -INFINITY;  // reference max of the row (log2 units)
      uint64_t l2 = pk2(0.f, 0.f);
      for (int j = 0; j < sl.n; ++j, ++g) {
        if (!warp_wait(bars + L::kSFull + s, g & 1, abort_flag, p.status)) { ok = false; break; }
        tc_fence_after_sync();
        uint32_t v[128];
#pragma unroll
        for (int q = 0; q < 4; ++q) VSA_TMEM_LD16(t_s + 16u * q, v, 16 * q);
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
        for (int q = 4; q < 8; ++q) VSA_TMEM_LD16(t_s + 16u * q, v, 16 * q);
        const int rem = limit - 128 * j;
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        const bool masked = __any_sync(0xffffffffu, rem < 128);
        if (masked) {
#pragma unroll
          for (int q = 0; q < 64; ++q)
            if (q >= rem) v[q] = __float_as_uint(-INFINITY);
        }
#pragma unroll
        for (int q = 0; q < 64; q += 8) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mx[e] = fmax3(mx[e], __uint_as_float(v[q + 2 * e]), __uint_as_float(v[q + 2 * e + 1]));
        }
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
        if (masked) {
#pragma unroll
          for (int q = 64; q < 128; ++q)
            if (q >= rem) v[q] = __float_as_uint(-INFINITY);
        }
#pragma unroll
        for (int q = 64; q < 128; q += 8) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mx[e] = fmax3(mx[e], __uint_as_float(v[q + 2 * e]), __uint_as_float(v[q + 2 * e + 1]));
        }
        const float top = fmax3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * c;
        const bool move = top > m + kRefresh;
        if (__any_sync(0xffffffffu, move)) {
          const float nm = move ? top : m;
          const float alpha = (m == -INFINITY) ? 0.f : fast_exp2(m - nm);
          float la, lb;
          upk2(l2, la, lb);
          l2 = pk2(la * alpha, lb * alpha);
          if (j > 0) {
            // rows that did not move have alpha = 1 (0 only while O is all zero)
            const float a = move ? alpha : 1.f;
#pragma unroll
            for (int q0 = 0; q0 < D; q0 += 16) {
              uint32_t ov[16];
              VSA_TMEM_LD16(t_o + q0, ov, 0);
              asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
              for (int q = 0; q < 16; ++q) ov[q] = __float_as_uint(__uint_as_float(ov[q]) * a);
              VSA_TMEM_ST16(t_o + q0, ov, 0);
            }
          }
          m = nm;
        }
        // probabilities 2^(s*c - m): bf16 pairs for the tensor core, fp32 sums
        const float ref = (m == -INFINITY) ? 0.f : -m;  // nothing seen yet: all -inf, all 0
        const uint64_t nm2 = pk2(ref, ref);
#pragma unroll
        for (int q0 = 0; q0 < 64; q0 += 16) {
          uint32_t pk[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            const int e = 2 * (q0 + q);
            float a, b;
            upk2(ffma2(pk2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), cc, nm2), a, b);
            uint64_t pp;
            if ((q & 7) < DENSE_POLY8) {
              // the clamp turns -inf into 2^-120; masked places must be 0
              pp = exp2_fma2_t<true>(a, b);
              if (masked) {
                float p0, p1;
                upk2(pp, p0, p1);
                pp = pk2(e < rem ? p0 : 0.f, e + 1 < rem ? p1 : 0.f);
              }
            } else {
              pp = pk2(fast_exp2(a), fast_exp2(b));
            }
            l2 = fadd2(l2, pp);
            float p0, p1;
            upk2(pp, p0, p1);
            pk[q] = pack_bf16x2(p0, p1);
          }
          VSA_TMEM_ST16(t_s + q0, pk, 0);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + L::kPFull + s);
      }
      if (!ok) break;
      // hand 1 / l to the epilogue, once it has taken the previous item's
      if (n >= 1 && !warp_wait(bars + L::kOEmpty + s, (n - 1) & 1, abort_flag, p.status)) { ok = false; break; }
      ++n;
      float la, lb;
      upk2(l2, la, lb);
      const float l = la + lb;
      inv_l[s * 128 + row] = l == 0.f ? 0.f : 1.f / l;
      if (p.lse && row < sl.rows)
        p.lse[sl.head * p.lse_seq + sl.row0 + row] =
            l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + L::kLFull + s);
    }
  } else {
    regs_dec<kRegsEpilogue>();
    // ===================== epilogue: one thread per query row =====================
    const int wq = warp - 12;
    const int row = wq * 32 + lane;
    const uint32_t t_lane = tmem_base + (uint32_t(wq * 32) << 16) + kTmemO;
    uint32_t cs[2] = {0, 0};
    bool ok = true;
    for (int w = 0, it; ok && (it = wave_item(w, cta, grid), w * grid < p.n_work); ++w) {
      if (it >= p.n_work) continue;
      const Item x = load_item(p, seqs, it);
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {
        // the shorter slot (1) ends first where the two differ
        const int s = x.n1 < x.n0 ? 1 - k : k;
        const Slot sl = get_slot(p, x, s);
        if (sl.rows == 0) continue;
        __nv_bfloat16* orow = p.out + sl.head * p.out_st.h + (long long)(sl.row0 + row) * p.out_st.s;
        const bool real = row < sl.rows;
        if (sl.n == 0) {
          // rows that see no key
          if (real) {
#pragma unroll
            for (int e = 0; e < D; e += 8) *reinterpret_cast<uint4*>(orow + e) = make_uint4(0u, 0u, 0u, 0u);
            if (p.lse) p.lse[sl.head * p.lse_seq + sl.row0 + row] = -INFINITY;
          }
          continue;
        }
        const uint32_t ph = cs[s] & 1;
        ++cs[s];
        if (!warp_wait(bars + L::kLFull + s, ph, abort_flag, p.status) ||
            !warp_wait(bars + L::kOFull + s, ph, abort_flag, p.status)) { ok = false; break; }
        tc_fence_after_sync();
        const float il = inv_l[s * 128 + row];
#pragma unroll
        for (int q0 = 0; q0 < D; q0 += 32) {
          uint32_t ov[32];
          tmem_ld32(t_lane + D * s + q0, ov);
          if (q0 + 32 == D) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars + L::kOEmpty + s);
          }
          if (real) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t o[4];
#pragma unroll
              for (int q = 0; q < 4; ++q)
                o[q] = pack_bf16x2(__uint_as_float(ov[e + 2 * q]) * il,
                                   __uint_as_float(ov[e + 2 * q + 1]) * il);
              *reinterpret_cast<uint4*>(orow + q0 + e) = make_uint4(o[0], o[1], o[2], o[3]);
            }
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
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  if (!cached[dev]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    cached[dev] = n;
  }
  return cached[dev];
}

int KernelReady::check(const void* kern, int regs, int smem) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return VSA_ERR_CUDA;
  const unsigned long long bit = 1ull << dev;
  if (done.load(std::memory_order_acquire) & bit) return VSA_OK;
  // a warpgroup's register increase could never be granted if the kernel had
  // been compiled to fewer registers than its split adds up to
  cudaFuncAttributes attr;
  if (cudaFuncGetAttributes(&attr, kern) != cudaSuccess) return VSA_ERR_CUDA;
  if (regs > 0 && attr.numRegs != regs) return VSA_ERR_UNSUPPORTED;
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

void fill_dense_seqs(DenseSeqs* t, const int4* seqs, const int* units, int n) {
  int order[kDenseMaxSeqs];
  int m = 0;
  for (int i = 0; i < n; ++i)
    if (units[i] > 0) order[m++] = i;
  std::stable_sort(order, order + m, [&](int a, int b) { return units[a] > units[b]; });
  t->n = m;
  for (int r = 0; r < m; ++r) {
    t->seq[r] = seqs[order[r]];
    t->units[r] = units[order[r]];
  }
  int items = 0;
  t->first[0] = 0;
  for (int r = 1; r <= m; ++r) {
    t->first[r] = items;
    items += r * (t->units[r - 1] - (r < m ? t->units[r] : 0));
  }
  t->first[m + 1] = items;
  t->n_items = items;
}

template <int D>
static int launch_dense_fwd_t(DenseParams p, const DenseSeqs& seqs, const CUtensorMap& mq,
                              const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t stream) {
  using L = dense::Layout<D>;
  auto kern = dense::dense_fwd_kernel<D>;
  static KernelReady ready;
  const int rc = ready.check(reinterpret_cast<const void*>(kern), (int)dense::kLaunchRegs, (int)L::kAlloc);
  if (rc != VSA_OK) return rc;
  p.n_work = seqs.n_items * p.Hkv;
  if (p.n_work == 0) return VSA_OK;
  const int sms = device_sm_count();
  const int grid = p.n_work < sms ? p.n_work : sms;
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
  for (int i0 = 0; i0 < b.n; i0 += kDenseMaxSeqs) {
    int4 seqs[kDenseMaxSeqs];
    int units[kDenseMaxSeqs];
    const int n = b.chunk(i0, seqs);
    long long slots = 0;
    for (int i = 0; i < n; ++i) slots += (seqs[i].y + 127LL) / 128 * p.Hq;
    if (slots >= (1 << 30)) return VSA_ERR_UNSUPPORTED;  // 32-bit item index
    // Two row tiles per item halve the K/V reads and let one slot's softmax run
    // under the other's products; with no more row tiles than SMs one tile per
    // item spreads them over twice as many SMs instead.
    p.slots = slots > device_sm_count() ? 2 : 1;
    for (int i = 0; i < n; ++i)
      units[i] = ((seqs[i].y + 127) / 128 * p.group + p.slots - 1) / p.slots;
    DenseSeqs table;
    fill_dense_seqs(&table, seqs, units, n);
    const int rc = D == 128 ? launch_dense_fwd_t<128>(p, table, mq, mk, mv, stream)
                            : launch_dense_fwd_t<64>(p, table, mq, mk, mv, stream);
    if (rc != VSA_OK) return rc;
  }
  return VSA_OK;
}

}  // namespace vsa

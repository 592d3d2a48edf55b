// Dense softmax attention over packed sequences with grouped heads, causal or
// full: the gradients.
//
// What it computes, per sequence and query head h (key head h / G), from the
// forward's out and lse (row r sees its first n(r) keys, see dense_fwd.cu):
//   p(r, j) = exp(scale q_r . k_j - lse(r))          (0 for j >= n(r))
//   delta(r) = sum_d dout(r, d) out(r, d)
//   ds(r, j) = p(r, j) (dout_r . v_j - delta(r))
//   dq_r = scale sum_j ds(r, j) k_j
//   dk_j = scale sum_{h, r} ds(r, j) q_r             (over the heads of the group)
//   dv_j = sum_{h, r} p(r, j) dout_r
//
// How (sm_100a): two kernels, each with one kind of accumulator in TMEM, so
// that every sum has one owner and a fixed order (no atomics).  The price is
// that S and dout V^T are formed twice (7 products of 128 x 128 x D instead of
// 5).  One kernel for all five was estimated, not built: it would send its dq
// tiles to memory as fp32 sums, 64 KB per pair of tiles each way through shared
// memory, and keep dS there too, some 3800 cycles of shared-memory traffic (128
// bytes a cycle) per pair of tiles, against the 4700 cycles that these seven
// products take; the key tiles that add to a query tile would have to take turns
// for the sums to keep their order.
//
//  dq:     a work item is one 128-row query tile of one head.  Per key tile
//            S = Q K^T, dP = dO V^T, dQ += dS K
//          Q, dO (bf16) and dS are A operands in TMEM, so only K and V tiles
//          are read from shared memory.
//  dk/dv:  a work item is one 128-row key tile of one key head; it walks the
//          query tiles of all heads of the group that see it.  Per query tile
//            S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q
//          P^T and dS^T are A operands in TMEM, over their own S and dP.  Where
//          key tiles are too few, several items share a tile's walk, leave fp32
//          sums, and a third kernel adds them up in order.
//
// Both: one CTA per SM, item after item, 768 threads: warp 0 tile loads, warp 1
// products (one thread), warps 2-3 helpers, warps 4-19 softmax (32 of the 128
// columns each), warps 20-23 epilogue.  Products are issued in pairs, dQ(j) with
// dP(j+1), and dV(i) with S(i+1), dK(i) with dP(i+1), after everything that
// both need was waited for: the thread's waits cost 100-250 cycles each, and a
// product's completion reaches a waiting warp 300 cycles after its last
// multiplication.  The exponentials of a tile run under one pair, its dS under
// the other (dq: under the next S).  dP of the dq kernel comes in halves of 64
// keys, so that the first half's dS runs under the second, and dQ begins with it.
//
// What bounds it at D = 128: a product of 128 x 128 x 128 takes 596 cycles with
// its A operand in TMEM, 861 with it in shared memory (A's 4 KB per instruction
// do not load under the multiplication), so dq has 3 x 596 = 1788 cycles a tile
// and dk/dv 2 x 596 + 2 x 861 = 2914 (TMEM holds no K and V beside two sums of
// 128 columns).  Measured on 8192 rows, 40 heads over 8: 2455 and 3290 cycles of
// the launch for each of an SM's pairs of tiles (start, end and the half-empty
// tiles on the diagonal included), 1.91 ms together, 900 TFLOP/s of the five
// products, at 1.7 GHz; called back to back, under the power limit, 2.19 ms.
// P and dS are rounded to bf16 for the tensor core; everything else is fp32.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "dense_attn.cuh"
#include "dense_launch.h"
#include "vsa.h"
#include "vsa_device.cuh"

namespace vsa {
namespace dense {
namespace {

using slim::mbar_wait;
using slim::warp_wait;

constexpr int kThreads = 768;
constexpr int kSoftmaxWarps = 16;
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2 = 1.4426950408889634f;
// 0 / 1 / 2 / 3: 1943, 1909, 1907, 1930 us on 8192 rows, 40 heads over 8; 764, 756,
// 756, 764 on seven documents of 8192 rows together, 56 over 8
#ifndef DENSE_BWD_POLY8
#define DENSE_BWD_POLY8 2  // column pairs in eight whose exponential runs on the FMA pipe
#endif

__device__ __forceinline__ uint32_t sw128(uint32_t row, uint32_t chunk) {
  return row * 128u + ((chunk ^ (row & 7u)) << 4);
}

// D = A B^T over N rows of B from its row `from` on: A [128][D] bf16 in TMEM, B a
// tile [D / 64][128 rows][128 B].
template <int D, int N>
__device__ __forceinline__ void issue_ta(uint32_t tmem_d, uint32_t tmem_a, uint32_t b_base, int from) {
  constexpr uint32_t idesc = make_idesc_bf16(128, N, false, false);
  const uint64_t b0 = make_sdesc_sw128(b_base + 128u * from, 16u, 1024u);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
    umma_bf16_tmem_a(tmem_d + from, tmem_a + 8u * kk,
                     b0 + (uint64_t)(((kk / 4) * 16384 + (kk % 4) * 32) >> 4), idesc, kk > 0 ? 1u : 0u);
}

// D (+)= A B over the steps [from, to) of 16 rows of the tile B [D / 64][128][128 B]
// (FROM, TO, and no further than `steps`); A [128][128] bf16 in TMEM: 32 columns at each of tmem_a + 0, 32, 64, 96 (over
// the fp32 columns of the softmax warpgroup that wrote them).
template <int D, int FROM, int TO>
__device__ __forceinline__ void issue_quarters(uint32_t tmem_d, uint32_t tmem_a, uint32_t b_base, int steps,
                                               bool accumulate) {
  constexpr uint32_t idesc = make_idesc_bf16(128, D, false, true);
  const uint64_t b0 = make_sdesc_sw128(b_base, 16384u, 1024u);
  if (steps >= TO) {
#pragma unroll
    for (int kk = FROM; kk < TO; ++kk)
      umma_bf16_tmem_a(tmem_d, tmem_a + 32u * (kk / 2) + 8u * (kk % 2), b0 + (uint64_t)((kk * 2048) >> 4),
                       idesc, (accumulate || kk > 0) ? 1u : 0u);
  } else {
    for (int kk = FROM; kk < steps; ++kk)
      umma_bf16_tmem_a(tmem_d, tmem_a + 32u * (kk / 2) + 8u * (kk % 2), b0 + (uint64_t)((kk * 2048) >> 4),
                       idesc, (accumulate || kk > 0) ? 1u : 0u);
  }
}

// 16 TMEM lanes x 16 columns of 32 bits: register 2 i + b holds lane
// threadIdx / 4 + 8 b, column 4 i + threadIdx % 4.
__device__ __forceinline__ void tmem_st_16x128(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// ---------------------------------------------------------------------------
// dq
// ---------------------------------------------------------------------------
struct QItem {
  int head, hk;
  int row0, rows;  // rows of q
  int kv0, kv_len;
  int lim0;        // keys that tile row 0 sees (causal: row r sees lim0 + r, may be <= 0)
  int last;        // keys that the last real row sees
  int n;           // key tiles
};

using QItems = ItemRing<QItem, 2>;

template <int D>
struct QLayout {
  static constexpr int DH = D / 64;
  static constexpr uint32_t kTile = 128u * D * 2u;
  static constexpr int NST = D == 128 ? 7 : 12;  // ring: Q, dO, out, K(0), V(0), K(1), ...
  static constexpr uint32_t kRingOff = 0;
  static constexpr uint32_t kRowOff = kRingOff + NST * kTile;  // [2][2][128] f32: -lse, delta
  static constexpr uint32_t kItemOff = kRowOff + 2048u;
  static constexpr uint32_t kBarOff = kItemOff + (uint32_t)sizeof(QItems);
  // Q, and dO with out, signal barriers of their item's, K and V tiles their
  // stage's.  Four of the former: the ring holds those of fewer than four items
  // ahead of the one whose operands are being copied.
  static constexpr int NOP = 4;
  static_assert(NST <= 5 * (NOP - 1), "an item takes five stages or more");
  static constexpr int kFull = 0, kEmpty = NST, kPre = 2 * NST, kQFull = 3 * NST,
                       kGFull = kQFull + NOP, kQReady = kGFull + NOP, kGReady = kQReady + 2,
                       kDReady = kGReady + 1, kQFree = kDReady + 2, kGFree = kQFree + 1,
                       kSFull = kGFree + 1, kSFree = kSFull + 1,
                       kDPFull = kSFree + 1, kDSFull = kDPFull + 2, kOFull = kDSFull + 2,
                       kOEmpty = kOFull + 1, kItFull = kOEmpty + 1, kItEmpty = kItFull + QItems::kSlots,
                       kTake = kItEmpty + QItems::kSlots, kLoaded = kTake + 1, kNumBars = kLoaded + 1;
  static constexpr uint32_t kMiscOff = kBarOff + 8u * kNumBars;
  static constexpr uint32_t kTakeOff = (kMiscOff + 16u + 15u) & ~15u;
  static constexpr uint32_t kAlloc = kTakeOff + 16u;
  static_assert(kAlloc <= 227u * 1024u, "shared memory");
};
// TMEM columns
constexpr uint32_t kQS = 0, kQDP = 128, kQDQ = 256, kQQ = 384, kQDO = 448;

__device__ __forceinline__ QItem load_qitem(const DenseBwdParams& p, const DenseSeqs& t, int w) {
  QItem x;
  x.hk = w % p.Hkv;
  const Unit un = find_unit(t, w / p.Hkv);
  const int4 q = t.seq[un.seq];
  const int tile = un.rank / p.group;
  x.head = x.hk * p.group + (un.rank - tile * p.group);
  x.row0 = q.x + 128 * tile;
  x.rows = min(128, q.y - 128 * tile);
  x.kv0 = q.z;
  x.kv_len = q.w;
  x.lim0 = p.causal ? q.w - q.y + 128 * tile + 1 : q.w;
  x.last = p.causal ? max(0, x.lim0 + x.rows - 1) : q.w;
  x.n = (x.last + 127) >> 7;
  return x;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    dense_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                    const __grid_constant__ CUtensorMap tm_o, const __grid_constant__ DenseBwdParams p, const __grid_constant__ DenseSeqs seqs) {
  using L = QLayout<D>;
  constexpr int NST = L::NST;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {  // the tiles' swizzle needs it; there is no room to align by hand
    set_status(p.status, VSA_ERR_UNSUPPORTED);
    return;
  }
  float* rowv = reinterpret_cast<float*>(smem + L::kRowOff);
  QItems* items = reinterpret_cast<QItems*>(smem + L::kItemOff);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);

  const int tid = threadIdx.x;
  const int warp = tid / 32, lane = tid % 32;

  // the first item takes a search in memory: before all else
  QItem first = {};
  if (warp == 3) first = load_qitem(p, seqs, blockIdx.x);

  if (warp == 0) {
    for (int i = lane; i < L::kNumBars; i += 32) {
      // a TMA transaction, a commit or one thread's arrival, except where the
      // epilogue's four or the softmax's eight warps arrive
      const uint32_t count = ((i >= L::kQReady && i < L::kQFree) || i == L::kOEmpty) ? 4u
                             : i == L::kSFree                                         ? (uint32_t)kSoftmaxWarps
                             : (i >= L::kDSFull && i < L::kOFull)                     ? kSoftmaxWarps / 2u
                             : (i >= L::kItEmpty && i < L::kTake)                                     ? kThreads / 32 - 1u  // all warps but one
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
    tma_prefetch_desc(&tm_do);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  auto next = [&](uint32_t& w, QItem& x) {
    return get_item(items, bars + L::kItFull, bars + L::kItEmpty, w, x, lane, abort_flag, p.status);
  };

  if (warp < 4) {
    if (warp == 0) {
      // ===================== tile loads =====================
      const uint64_t keep = l2_policy_evict_last(), once = l2_policy_evict_first();
      uint32_t g = 0, n_item = 0;
      bool ok = true;
      QItem x;
      while (ok && next(n_item, x)) {
        if (lane == 0) {
          for (int j = -3; ok && j < 2 * x.n; ++j, ++g) {
            const int st = (int)(g % NST);
            const uint32_t u = g / NST;
            if (u >= 1) ok = mbar_wait(bars + L::kEmpty + st, (u - 1) & 1, abort_flag, p.status);
            if (!ok) break;
            uint8_t* dst = smem + L::kRingOff + st * L::kTile;
            const int key = 128 * (j >> 1);
            const bool is_v = j & 1;
            // a K tile with rows past the sequence goes through warp 2 first
            uint64_t* full = bars + (j < 0 ? (j == -3 ? L::kQFull : L::kGFull) + (int)((n_item - 1) % L::NOP)
                                           : (!is_v && x.kv_len - key < 128 ? L::kPre : L::kFull) + st);
            if (j != -1) mbar_arrive_expect_tx(full, j == -2 ? 2 * L::kTile : L::kTile);
#pragma unroll
            for (int dh = 0; dh < L::DH; ++dh) {
              uint8_t* to = dst + dh * 16384;
              if (j < 0)
                load_rows(to, j == -3 ? &tm_q : j == -2 ? &tm_do : &tm_o,
                          j == -3 ? p.q_ax : j == -2 ? p.do_ax : p.o_ax, full, dh * 64, x.row0, x.head, 0, once);
              else
                load_rows(to, is_v ? &tm_v : &tm_k, is_v ? p.v_ax : p.k_ax, full, dh * 64, x.kv0 + key, x.hk, 0, keep);
            }
          }
          mbar_arrive(bars + L::kLoaded);
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      }
      __syncwarp();
    } else if (warp == 3) {
      // ===================== work items; rows that see no key =====================
      uint32_t n_item = 0;
      bool ok = true;
      QItem x = first;
      Takeover take{bars + L::kTake, reinterpret_cast<uint4*>(smem + L::kTakeOff), 0};
      for (int it = blockIdx.x; ok && it >= 0; it = ok ? take.answer(abort_flag, p.status) : -1) {
        if (it != (int)blockIdx.x) x = load_qitem(p, seqs, it);
        if (x.n > 0) {
          // ask for more when this item's last tiles are on their way, not earlier:
          // what a CTA holds no other can take
          ok = put_item(items, bars + L::kItFull, bars + L::kItEmpty, n_item, x, lane, abort_flag, p.status) &&
               warp_wait(bars + L::kLoaded, n_item & 1, abort_flag, p.status);
          ++n_item;
          if (ok) take.ask(lane);
          continue;
        }
        take.ask(lane);
        for (int r = lane; r < x.rows; r += 32) {
          __nv_bfloat16* to = p.dq + x.head * p.dq_st.h + (long long)(x.row0 + r) * p.dq_st.s;
          for (int e = 0; e < D; e += 8) *reinterpret_cast<uint4*>(to + e) = make_uint4(0u, 0u, 0u, 0u);
          p.delta[x.head * p.lse_seq + x.row0 + r] = 0.f;
        }
      }
      x.n = -1;
      if (ok) put_item(items, bars + L::kItFull, bars + L::kItEmpty, n_item, x, lane, abort_flag, p.status);
    } else if (warp == 2) {
      // ===================== zero K rows past a sequence's keys (0 * inf is not 0) =====================
      uint32_t g = 0, pre = 0, n_item = 0;
      QItem x;
      while (next(n_item, x)) {
        g += 2 * x.n + 3;
        const int len = x.kv_len - 128 * (x.n - 1);
        if (len >= 128) continue;
        const int st = (int)((g - 2) % NST);
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
        uint32_t phase = 0;          // phase bit per ring stage
        uint32_t ts = 0, tq = 0;     // S and dQ products so far
        uint32_t n_s = 0, n_dp = 0;  // items whose first S, first dP was issued
        uint32_t g = 0, n_got = 0, n_item = 0;
        bool ok = true;
        auto wait = [&](int bar, uint32_t ph) {
          if (!mbar_wait(bars + bar, ph & 1, abort_flag, p.status)) ok = false;
        };
        auto wait_stage = [&](uint32_t at) {
          const uint32_t st = at % NST;
          wait(L::kFull + (int)st, phase >> st);
          phase ^= 1u << st;
        };
        auto tile = [&](uint32_t at) { return sbase + L::kRingOff + (at % NST) * L::kTile; };
        auto release = [&](uint32_t at) { mbar_arrive(bars + L::kEmpty + (int)(at % NST)); };
        // S(j) of item x, whose ring tiles start at gx
        auto do_s = [&](const QItem& x, int j, uint32_t gx) {
          if (j == 0) {
            // Q is in TMEM, its ring stage free again
            wait(L::kQReady + (int)(n_s & 1), n_s >> 1);
            ++n_s;
            release(gx);
          }
          wait_stage(gx + 3 + 2 * j);
          if (ts >= 1) wait(L::kSFree, ts - 1);
          if (!ok) return;
          ++ts;
          tc_fence_after_sync();
          issue_ta<D, 128>(tmem_base + kQS, tmem_base + kQQ, tile(gx + 3 + 2 * j), 0);
          umma_commit(bars + L::kSFull);
          if (j == x.n - 1) umma_commit(bars + L::kQFree);
        };
        // what dP(j) waits for, and dP(j)
        auto before_dp = [&](int j, uint32_t gx) {
          if (j == 0) wait(L::kGReady, n_dp++);
          wait_stage(gx + 4 + 2 * j);
        };
        auto do_dp = [&](const QItem& x, int j, uint32_t gx) {
          issue_ta<D, 64>(tmem_base + kQDP, tmem_base + kQDO, tile(gx + 4 + 2 * j), 0);
          umma_commit(bars + L::kDPFull);
          issue_ta<D, 64>(tmem_base + kQDP, tmem_base + kQDO, tile(gx + 4 + 2 * j), 64);
          umma_commit(bars + L::kDPFull + 1);
          if (j == x.n - 1) umma_commit(bars + L::kGFree);
        };
        auto next_one = [&](QItem& x) {
          return get_item_one(items, bars + L::kItFull, bars + L::kItEmpty, n_got, x, abort_flag, p.status);
        };
        QItem x, y;
        bool have = next_one(x);
        if (have) {
          do_s(x, 0, 0);
          before_dp(0, 0);
          tc_fence_after_sync();
          if (ok) do_dp(x, 0, 0);
        }
        while (ok && have) {
          bool more = false;
          const uint32_t g_next = g + 2 * x.n + 3;
          // delta is formed: dO and out are read.  Released here, before the next
          // item's first S: with one key tile the ring cannot take that item's K
          // until then.
          wait(L::kDReady + (int)(n_item & 1), n_item >> 1);
          if (!ok) break;
          release(g + 1);
          release(g + 2);
          for (int j = 0; ok && j < x.n; ++j) {
            const bool last = j + 1 == x.n;
            // (the item's tiles are all here, so that the next one was asked for)
            if (last) more = next_one(y);
            if (!last) do_s(x, j + 1, g);
            else if (more) do_s(y, 0, g_next);
            // everything that dP will need first, so that it follows dQ at once
            if (!last) before_dp(j + 1, g);
            else if (more) before_dp(0, g_next);
            // the epilogue has taken the previous item's dQ
            if (j == 0 && n_item >= 1) wait(L::kOEmpty, n_item - 1);
            wait(L::kDSFull, tq);
            ++tq;
            if (!ok) break;
            tc_fence_after_sync();
            const int keys = x.last - 128 * j;
            const int steps = keys >= 128 ? 8 : (keys + 15) >> 4;
            issue_quarters<D, 0, 4>(tmem_base + kQDQ, tmem_base + kQDP, tile(g + 3 + 2 * j), steps, j > 0);
            wait(L::kDSFull + 1, tq - 1);
            if (!ok) break;
            tc_fence_after_sync();
            issue_quarters<D, 4, 8>(tmem_base + kQDQ, tmem_base + kQDP, tile(g + 3 + 2 * j), steps, j > 0);
            if (last) umma_commit(bars + L::kOFull);
            if (!last) do_dp(x, j + 1, g);
            else if (more) do_dp(y, 0, g_next);
          }
          g = g_next;
          x = y;
          have = more;
          ++n_item;
        }
      }
      __syncwarp();
    }
  } else if (warp < 4 + kSoftmaxWarps) {
    // ===================== p and ds: one thread per query row and 32 keys =====================
    const int quarter = (warp - 4) >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t t_lane = tmem_base + (uint32_t((warp & 3) * 32) << 16) + 32u * quarter;
    const uint64_t cc = pk2(p.scale_log2, p.scale_log2);
    uint32_t g = 0, n_item = 0, n_got = 0;
    uint32_t at = 0, last_k = 0;  // ring tiles before the item; the previous key tile's K
    bool ok = true;
    QItem x;
    while (ok && next(n_got, x)) {
      if (!warp_wait(bars + L::kQReady + (n_item & 1), (n_item >> 1) & 1, abort_flag, p.status)) break;
      const float nl = rowv[(n_item & 1) * 256 + row];
      const uint64_t nl2 = pk2(nl, nl);
      uint64_t nd2 = 0;
      const int limit = p.causal ? min(x.lim0 + row, x.kv_len) : x.kv_len;  // keys this row sees
      for (int j = 0; j < x.n; ++j, ++g) {
        if (!warp_wait(bars + L::kSFull, g & 1, abort_flag, p.status)) { ok = false; break; }
        tc_fence_after_sync();
        uint32_t v[32];
        tmem_ld32(t_lane + kQS, v);
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + L::kSFree);
        const int rem = limit - 128 * j - 32 * quarter;
        const bool masked = __any_sync(0xffffffffu, rem < 32);
        auto probs = [&](auto mask) {
          constexpr bool kMask = decltype(mask)::value;
          if (kMask) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e >= rem) v[e] = __float_as_uint(-INFINITY);
          }
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const uint64_t e = ffma2(pk2(__uint_as_float(v[2 * q]), __uint_as_float(v[2 * q + 1])), cc, nl2);
          float a, b;
          upk2(e, a, b);
          if (!kMask && (q & 7) < DENSE_BWD_POLY8) {
            upk2(exp2_fma2_any(a, b), a, b);
          } else {
            a = fast_exp2(a);
            b = fast_exp2(b);
          }
          v[2 * q] = __float_as_uint(a);
          v[2 * q + 1] = __float_as_uint(b);
        }
        };
        if (masked) probs(std::true_type{});
        else probs(std::false_type{});
        if (j == 0) {
          if (!warp_wait(bars + L::kDReady + (n_item & 1), (n_item >> 1) & 1, abort_flag, p.status)) { ok = false; break; }
          const float nd = -rowv[(n_item & 1) * 256 + 128 + row];
          nd2 = pk2(nd, nd);
        }
        if (!warp_wait(bars + L::kDPFull + (quarter >> 1), g & 1, abort_flag, p.status)) { ok = false; break; }
        tc_fence_after_sync();
        if (warp == 12 && lane == 0) {
          // dP's second half is complete, and with it all before it: its V tile and the
          // previous dQ's K tile are free
          mbar_arrive(bars + L::kEmpty + (int)((at + 4 + 2 * j) % NST));
          if (g > 0) mbar_arrive(bars + L::kEmpty + (int)(last_k % NST));
          last_k = at + 3 + 2 * j;
        }
        uint32_t dp[32], pk[16];
        tmem_ld32(t_lane + kQDP, dp);
        if (masked) {
          // p = 0 there, but dP may be infinite
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (e >= rem) dp[e] = 0u;
        }
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          float a, b;
          upk2(fmul2(fadd2(pk2(__uint_as_float(dp[2 * q]), __uint_as_float(dp[2 * q + 1])), nd2),
                     pk2(__uint_as_float(v[2 * q]), __uint_as_float(v[2 * q + 1]))), a, b);
          pk[q] = pack_bf16x2(a, b);
        }
        // over columns that this thread has read
        VSA_TMEM_ST16(t_lane + kQDP, pk, 0);
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + L::kDSFull + (quarter >> 1));
      }
      ++n_item;
      at += 2 * x.n + 3;
    }
  } else {
    // ===================== operands, delta and results: one thread per query row =====================
    const int row = (warp & 3) * 32 + lane;
    const uint32_t t_lane = tmem_base + (uint32_t((warp & 3) * 32) << 16);
    uint32_t g = 0, n_item = 0;
    bool ok = true;
    QItem prev = {};
    auto read_out = [&](const QItem& x, uint32_t idx) {
      if (!warp_wait(bars + L::kOFull, idx & 1, abort_flag, p.status)) return false;
      tc_fence_after_sync();
      __nv_bfloat16* to = p.dq + x.head * p.dq_st.h + (long long)(x.row0 + row) * p.dq_st.s;
#pragma unroll 1
      for (int q0 = 0; q0 < D; q0 += 32) {
        uint32_t ov[32];
        tmem_ld32(t_lane + kQDQ + q0, ov);
        if (q0 + 32 == D) {
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(bars + L::kOEmpty);
        }
        if (row < x.rows) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t o[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              o[q] = pack_bf16x2(__uint_as_float(ov[e + 2 * q]) * p.scale,
                                 __uint_as_float(ov[e + 2 * q + 1]) * p.scale);
            *reinterpret_cast<uint4*>(to + q0 + e) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      }
      return true;
    };
    uint32_t n_got = 0;
    QItem x;
    while (ok && next(n_got, x)) {
      const bool real = row < x.rows;
      const float lse = real ? p.lse[x.head * p.lse_seq + x.row0 + row] : 0.f;
      const uint32_t sq = g % NST, sd = (g + 1) % NST, so = (g + 2) % NST;
      const uint8_t* qt = smem + L::kRingOff + sq * L::kTile;
      const uint8_t* dt = smem + L::kRingOff + sd * L::kTile;
      const uint8_t* ot = smem + L::kRingOff + so * L::kTile;
      const bool sees = lse != -INFINITY;  // else all of the row is masked
      rowv[(n_item & 1) * 256 + row] = sees ? -lse * kLog2 : 0.f;
      // this thread's row of a tile -> bf16 A operand in TMEM
      auto copy_row = [&](const uint8_t* tile, uint32_t col) {
#pragma unroll 1
        for (int c0 = 0; c0 < D / 8; c0 += 8) {
          uint32_t a[32];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint4 x4 = *reinterpret_cast<const uint4*>(tile + (c0 >> 3) * 16384 + sw128(row, c));
            a[4 * c] = x4.x, a[4 * c + 1] = x4.y, a[4 * c + 2] = x4.z, a[4 * c + 3] = x4.w;
          }
          VSA_TMEM_ST16(t_lane + col + 4 * c0, a, 0);
          VSA_TMEM_ST16(t_lane + col + 4 * c0 + 16, a, 16);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before_sync();
        __syncwarp();
      };
      // Q, once the previous item's last S is complete
      if (!warp_wait(bars + L::kQFull + (int)(n_item % L::NOP), (n_item / L::NOP) & 1, abort_flag, p.status) ||
          (n_item >= 1 && !warp_wait(bars + L::kQFree, (n_item - 1) & 1, abort_flag, p.status))) break;
      tc_fence_after_sync();
      copy_row(qt, kQQ);
      if (lane == 0) mbar_arrive(bars + L::kQReady + (n_item & 1));
      // dO, once its last dP is
      if (!warp_wait(bars + L::kGFull + (int)(n_item % L::NOP), (n_item / L::NOP) & 1, abort_flag, p.status) ||
          (n_item >= 1 && !warp_wait(bars + L::kGFree, (n_item - 1) & 1, abort_flag, p.status))) break;
      tc_fence_after_sync();
      copy_row(dt, kQDO);
      if (lane == 0) mbar_arrive(bars + L::kGReady);
      float delta = 0.f;
#pragma unroll 4
      for (int ch = 0; ch < D / 8; ++ch) {
        const uint32_t off = (ch >> 3) * 16384 + sw128(row, ch & 7);
        const uint4 o4 = *reinterpret_cast<const uint4*>(ot + off);
        const uint4 d4 = *reinterpret_cast<const uint4*>(dt + off);
        const __nv_bfloat162* o2 = reinterpret_cast<const __nv_bfloat162*>(&o4);
        const __nv_bfloat162* d2 = reinterpret_cast<const __nv_bfloat162*>(&d4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 a = __bfloat1622float2(o2[e]), c = __bfloat1622float2(d2[e]);
          delta = fmaf(a.x, c.x, delta);
          delta = fmaf(a.y, c.y, delta);
        }
      }
      if (!sees) delta = 0.f;
      rowv[(n_item & 1) * 256 + 128 + row] = delta;
      if (real) p.delta[x.head * p.lse_seq + x.row0 + row] = delta;
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + L::kDReady + (n_item & 1));
      if (n_item >= 1 && !read_out(prev, n_item - 1)) { ok = false; break; }
      prev = x;
      g += 2 * x.n + 3;
      ++n_item;
    }
    if (ok && !abort_flag[0] && n_item >= 1) read_out(prev, n_item - 1);
  }

  settle_after_abort(abort_flag);
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// dk and dv
// ---------------------------------------------------------------------------
struct KItem {
  int hk;
  int key0, keys;  // rows of k
  int q0, q_len;   // first row of q that sees the tile, and the rows from there on
  int diag;        // causal: tile key i is seen by rows q0 + r with r + diag >= i
  int tiles;       // query tiles of one head
  int head0, t0;   // where the item's walk begins: head of the group, query tile
  int n;           // query tiles of the walk
  int part;        // which share of the tile's walk it is
};

using KItems = ItemRing<KItem, 2>;

template <int D>
struct KLayout {
  static constexpr int DH = D / 64;
  static constexpr uint32_t kTile = 128u * D * 2u;
  static constexpr int NST = D == 128 ? 5 : 10;  // ring: Q(0), dO(0), Q(1), ...
  static constexpr int NROW = 2;                // ring of -lse and delta rows
  static constexpr uint32_t kKOff = 0, kVOff = kTile;
  static constexpr uint32_t kRingOff = 2 * kTile;
  static constexpr uint32_t kRowOff = kRingOff + NST * kTile;  // [NROW][2][128] f32
  static constexpr uint32_t kItemOff = kRowOff + NROW * 1024u;
  static constexpr uint32_t kBarOff = kItemOff + (uint32_t)sizeof(KItems);
  static constexpr int kFull = 0, kEmpty = NST, kPre = 2 * NST, kRowFull = 3 * NST,
                       kRowEmpty = kRowFull + NROW, kKFull = kRowEmpty + NROW, kKEmpty = kKFull + 1,
                       kVFull = kKEmpty + 1, kVEmpty = kVFull + 1, kSFull = kVEmpty + 1, kPFull = kSFull + 1, kDPFull = kPFull + 1,
                       kDSFull = kDPFull + 1, kDVFull = kDSFull + 1, kDKFull = kDVFull + 1,
                       kDVEmpty = kDKFull + 1, kDKEmpty = kDVEmpty + 1, kItFull = kDKEmpty + 1, kItEmpty = kItFull + KItems::kSlots,
                       kTake = kItEmpty + KItems::kSlots, kLoaded = kTake + 1, kNumBars = kLoaded + 1;
  static constexpr uint32_t kMiscOff = kBarOff + 8u * kNumBars;
  static constexpr uint32_t kTakeOff = (kMiscOff + 16u + 15u) & ~15u;
  static constexpr uint32_t kAlloc = kTakeOff + 16u;
  static_assert(kAlloc <= 227u * 1024u, "shared memory");
};
constexpr uint32_t kKS = 0, kKDP = 128, kKDV = 256, kKDK = 384;

__device__ __forceinline__ KItem load_kitem(const DenseBwdParams& p, const DenseSeqs& t, int w) {
  KItem x;
  x.part = w % p.parts;
  w /= p.parts;
  x.hk = w % p.Hkv;
  const Unit un = find_unit(t, w / p.Hkv);
  const int4 q = t.seq[un.seq];
  // the first key tiles are seen by the most rows: longest first
  const int tile = t.units[un.seq] - 1 - un.rank;
  x.key0 = q.z + 128 * tile;
  x.keys = min(128, q.w - 128 * tile);
  const int off = q.w - q.y;
  const int skip = p.causal ? max(0, 128 * tile - off) : 0;
  x.q0 = q.x + skip;
  x.q_len = max(0, q.y - skip);
  x.diag = skip + off - 128 * tile;
  x.tiles = (x.q_len + 127) >> 7;
  // (the host keeps walks below 2^27 tiles)
  const int all = x.tiles * p.group, from = all * x.part / p.parts;
  x.n = all * (x.part + 1) / p.parts - from;
  x.head0 = x.tiles ? from / x.tiles : 0;
  x.t0 = from - x.head0 * x.tiles;
  return x;
}

// Row r of the item's key tile among the partial sums; dv's lie Hkv * part_rows
// rows after dk's.
template <int D>
__device__ __forceinline__ float* part_row(const DenseBwdParams& p, const KItem& x, int r) {
  return p.part + (((long long)x.part * 2 * p.Hkv + x.hk) * p.part_rows + (x.key0 - p.part_row0 + r)) * D;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    dense_dkv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                     const __grid_constant__ DenseBwdParams p, const __grid_constant__ DenseSeqs seqs) {
  using L = KLayout<D>;
  constexpr int NST = L::NST, NROW = L::NROW;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {  // the tiles' swizzle needs it; there is no room to align by hand
    set_status(p.status, VSA_ERR_UNSUPPORTED);
    return;
  }
  float* rowv = reinterpret_cast<float*>(smem + L::kRowOff);
  KItems* items = reinterpret_cast<KItems*>(smem + L::kItemOff);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);

  const int tid = threadIdx.x;
  const int warp = tid / 32, lane = tid % 32;

  // the first item takes a search in memory: before all else
  KItem first = {};
  if (warp == 2) first = load_kitem(p, seqs, blockIdx.x);

  if (warp == 0) {
    for (int i = lane; i < L::kNumBars; i += 32) {
      const uint32_t count = (i == L::kDVEmpty || i == L::kDKEmpty) ? 4u
                             : (i == L::kPFull || i == L::kDSFull ||
                                (i >= L::kRowEmpty && i < L::kRowEmpty + NROW)) ? (uint32_t)kSoftmaxWarps
                             : (i >= L::kItEmpty && i < L::kTake)                              ? kThreads / 32 - 1u  // all warps but one
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
    tma_prefetch_desc(&tm_do);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  auto next = [&](uint32_t& w, KItem& x) {
    return get_item(items, bars + L::kItFull, bars + L::kItEmpty, w, x, lane, abort_flag, p.status);
  };

  if (warp < 4) {
    if (warp == 0) {
      // ===================== Q and dO tiles =====================
      const uint64_t keep = l2_policy_evict_last();
      uint32_t g = 0, n_item = 0;
      bool ok = true;
      KItem x;
      while (ok && next(n_item, x)) {
        if (lane == 0) {
          int head = x.hk * p.group + x.head0, t = x.t0;
          for (int i = 0; ok && i < 2 * x.n; ++i, ++g) {
            const int st = (int)(g % NST);
            const uint32_t u = g / NST;
            if (u >= 1) ok = mbar_wait(bars + L::kEmpty + st, (u - 1) & 1, abort_flag, p.status);
            if (!ok) break;
            const bool is_do = i & 1;
            const int r = 128 * t;
            // a tile with rows past the sequence goes through warp 3 first
            uint64_t* full = bars + (x.q_len - r < 128 ? L::kPre : L::kFull) + st;
            uint8_t* dst = smem + L::kRingOff + st * L::kTile;
            mbar_arrive_expect_tx(full, L::kTile);
#pragma unroll
            for (int dh = 0; dh < L::DH; ++dh)
              load_rows(dst + dh * 16384, is_do ? &tm_do : &tm_q, is_do ? p.do_ax : p.q_ax, full, dh * 64,
                        x.q0 + r, head, 0, keep);
            if (is_do && ++t == x.tiles) {
              t = 0;
              ++head;
            }
          }
          mbar_arrive(bars + L::kLoaded);
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      }
      __syncwarp();
    } else if (warp == 2) {
      // ===================== work items, their K and V tiles; keys that no row sees =====================
      const uint64_t once = l2_policy_evict_first();
      uint32_t n_item = 0;
      bool ok = true;
      KItem x = first;
      Takeover take{bars + L::kTake, reinterpret_cast<uint4*>(smem + L::kTakeOff), 0};
      for (int it = blockIdx.x; ok && it >= 0; it = ok ? take.answer(abort_flag, p.status) : -1) {
        if (it != (int)blockIdx.x) x = load_kitem(p, seqs, it);
        if (x.n == 0) {
          take.ask(lane);
          for (int r = lane; r < x.keys; r += 32) {
            if (p.parts > 1) {
              float* to = part_row<D>(p, x, r);
              for (int e = 0; e < D; e += 4) {
                *reinterpret_cast<float4*>(to + e) = make_float4(0.f, 0.f, 0.f, 0.f);
                *reinterpret_cast<float4*>(to + (long long)p.Hkv * p.part_rows * D + e) = make_float4(0.f, 0.f, 0.f, 0.f);
              }
              continue;
            }
            __nv_bfloat16* tk = p.dk + x.hk * p.dk_st.h + (long long)(x.key0 + r) * p.dk_st.s;
            __nv_bfloat16* tv = p.dv + x.hk * p.dv_st.h + (long long)(x.key0 + r) * p.dv_st.s;
            for (int e = 0; e < D; e += 8) {
              *reinterpret_cast<uint4*>(tk + e) = make_uint4(0u, 0u, 0u, 0u);
              *reinterpret_cast<uint4*>(tv + e) = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          continue;
        }
        if (!put_item(items, bars + L::kItFull, bars + L::kItEmpty, n_item, x, lane, abort_flag, p.status)) { ok = false; break; }
        if (lane == 0) {
          // K, once the previous item's last S is complete; V, once its last dP is
          if (n_item >= 1) ok = mbar_wait(bars + L::kKEmpty, (n_item - 1) & 1, abort_flag, p.status);
          if (ok) {
            mbar_arrive_expect_tx(bars + L::kKFull, L::kTile);
#pragma unroll
            for (int dh = 0; dh < L::DH; ++dh)
              load_rows(smem + L::kKOff + dh * 16384, &tm_k, p.k_ax, bars + L::kKFull, dh * 64, x.key0, x.hk, 0, once);
            if (n_item >= 1) ok = mbar_wait(bars + L::kVEmpty, (n_item - 1) & 1, abort_flag, p.status);
          }
          if (ok) {
            mbar_arrive_expect_tx(bars + L::kVFull, L::kTile);
#pragma unroll
            for (int dh = 0; dh < L::DH; ++dh)
              load_rows(smem + L::kVOff + dh * 16384, &tm_v, p.v_ax, bars + L::kVFull, dh * 64, x.key0, x.hk, 0, once);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        // ask for more when this item's last tiles are on their way, not earlier:
        // what a CTA holds no other can take
        ok = ok && warp_wait(bars + L::kLoaded, n_item & 1, abort_flag, p.status);
        ++n_item;
        if (ok) take.ask(lane);
      }
      x.n = -1;
      if (ok) ok = put_item(items, bars + L::kItFull, bars + L::kItEmpty, n_item, x, lane, abort_flag, p.status);
      // every copy has been consumed before exit
      if (ok && lane == 0 && n_item >= 1) mbar_wait(bars + L::kVEmpty, (n_item - 1) & 1, abort_flag, p.status);
      __syncwarp();
    } else if (warp == 3) {
      // ============ -lse and delta rows; zero Q and dO rows past a sequence ============
      uint32_t g = 0, pre = 0, n_item = 0;  // query tiles so far; phase bit per ring stage; items
      bool ok = true;
      KItem x;
      while (ok && next(n_item, x)) {
        int head = x.hk * p.group + x.head0, t = x.t0;
        for (int i = 0; ok && i < x.n; ++i, ++g) {
          const long long at = head * p.lse_seq + x.q0 + 128 * t;
          const int slot = (int)(g % NROW);
          const int left = x.q_len - 128 * t;
          if (++t == x.tiles) {
            t = 0;
            ++head;
          }
          float nl[4], de[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = 32 * e + lane;
            const bool real = r < left;
            // no row, or one whose logits are all -inf: p = 0
            const float lse = real ? p.lse[at + r] : -INFINITY;
            nl[e] = lse == -INFINITY ? -INFINITY : -kLog2 * lse;
            de[e] = real ? p.delta[at + r] : 0.f;
          }
          if (g >= (uint32_t)NROW &&
              !warp_wait(bars + L::kRowEmpty + slot, (g / NROW - 1) & 1, abort_flag, p.status)) { ok = false; break; }
          float* to = rowv + slot * 256;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            to[32 * e + lane] = nl[e];
            to[128 + 32 * e + lane] = -de[e];
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bars + L::kRowFull + slot);
          if (left >= 128) continue;
#pragma unroll 1
          for (int s = 0; ok && s < 2; ++s) {
            const int st = (int)((2 * g + s) % NST);
            if (!warp_wait(bars + L::kPre + st, (pre >> st) & 1, abort_flag, p.status)) { ok = false; break; }
            pre ^= 1u << st;
            zero_rows<128>(smem + L::kRingOff + st * L::kTile, L::DH, left, (left + 15) & ~15, lane);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars + L::kFull + st);
          }
        }
      }
    } else {
      // ===================== MMA issue: one thread =====================
      if (elect_one()) {
        uint32_t g = 0;    // query tiles so far
        uint32_t n_s = 0, n_dp = 0;  // items whose first S, first dP was prepared
        uint32_t n_got = 0, n_item = 0;
        bool ok = true;
        auto wait = [&](int bar, uint32_t ph) {
          if (!mbar_wait(bars + bar, ph & 1, abort_flag, p.status)) ok = false;
        };
        auto wait_stage = [&](uint32_t at) { wait(L::kFull + (int)(at % NST), at / NST); };
        auto tile = [&](uint32_t at) { return sbase + L::kRingOff + (at % NST) * L::kTile; };
        // S of query tile number t and what it waits for (its i-th of item x)
        auto before_s = [&](int i, uint32_t t) {
          if (i == 0) wait(L::kKFull, n_s++);
          wait_stage(2 * t);
        };
        auto do_s = [&](const KItem& x, int i, uint32_t t) {
          issue_s<D>(tmem_base + kKS, sbase + L::kKOff, tile(2 * t));
          umma_commit(bars + L::kSFull);
          if (i == x.n - 1) umma_commit(bars + L::kKEmpty);
        };
        auto before_dp = [&](int i, uint32_t t) {
          if (i == 0) wait(L::kVFull, n_dp++);
          wait_stage(2 * t + 1);
        };
        auto do_dp = [&](const KItem& x, int i, uint32_t t) {
          issue_s<D>(tmem_base + kKDP, sbase + L::kVOff, tile(2 * t + 1));
          umma_commit(bars + L::kDPFull);
          if (i == x.n - 1) umma_commit(bars + L::kVEmpty);
        };
        auto next_one = [&](KItem& x) {
          return get_item_one(items, bars + L::kItFull, bars + L::kItEmpty, n_got, x, abort_flag, p.status);
        };
        KItem x, y;
        bool have = next_one(x);
        if (have) {
          before_s(0, 0);
          tc_fence_after_sync();
          if (ok) do_s(x, 0, 0);
          before_dp(0, 0);
          tc_fence_after_sync();
          if (ok) do_dp(x, 0, 0);
        }
        while (ok && have) {
          bool more = false;
          int t = x.t0;  // query tile of the head
          for (int i = 0; ok && i < x.n; ++i, ++g) {
            const bool last = i + 1 == x.n;
            const int left = x.q_len - 128 * t;
            const int steps = left >= 128 ? 8 : (left + 15) >> 4;
            if (++t == x.tiles) t = 0;
            // (the item's tiles are all here, so that the next one was asked for)
            if (last) more = next_one(y);
            // dV, then the next S: everything that S will need first, so that it follows at once
            if (!last || more) before_s(last ? 0 : i + 1, g + 1);
            // the epilogue has taken the previous item's dV
            if (i == 0 && n_item >= 1) wait(L::kDVEmpty, n_item - 1);
            wait(L::kPFull, g);
            if (!ok) break;
            tc_fence_after_sync();
            issue_quarters<D, 0, 8>(tmem_base + kKDV, tmem_base + kKS, tile(2 * g + 1), steps, i > 0);
            if (last) umma_commit(bars + L::kDVFull);
            if (!last) do_s(x, i + 1, g + 1);
            else if (more) do_s(y, 0, g + 1);
            // dK, then the next dP
            if (!last || more) before_dp(last ? 0 : i + 1, g + 1);
            if (i == 0 && n_item >= 1) wait(L::kDKEmpty, n_item - 1);
            wait(L::kDSFull, g);
            if (!ok) break;
            tc_fence_after_sync();
            issue_quarters<D, 0, 8>(tmem_base + kKDK, tmem_base + kKDP, tile(2 * g), steps, i > 0);
            umma_commit(bars + L::kEmpty + (int)((2 * g) % NST));
            if (last) umma_commit(bars + L::kDKFull);
            if (!last) do_dp(x, i + 1, g + 1);
            else if (more) do_dp(y, 0, g + 1);
          }
          x = y;
          have = more;
          ++n_item;
        }
      }
      __syncwarp();
    }
  } else if (warp < 4 + kSoftmaxWarps) {
    // ===================== p and ds =====================
    // A warp has 32 keys (TMEM lanes) and 32 query rows (columns).  -lse and
    // delta go with the columns, so they come from shared memory; a thread
    // that held one key's part of S would read 32 of each, and a warp's reads of
    // one address cost as much as reads of 32.  In the 16x256b form a thread
    // holds four keys (lane / 4 + 8 k) and the columns 8 i + 2 (lane % 4) + {0, 1}
    // and reads a quarter of that (8 warps of 64 columns: 1950 -> 1510 cycles for p).
    const int quarter = (warp - 4) >> 2;
    const uint32_t t_lane = tmem_base + (uint32_t((warp & 3) * 32) << 16) + 32u * quarter;
    constexpr uint32_t kUpper = 16u << 16;  // lanes 16-31 of the warp
    const int row0 = (warp & 3) * 32 + lane / 4, col0 = 2 * (lane & 3);
    const uint64_t cc = pk2(p.scale_log2, p.scale_log2);
    uint32_t g = 0, n_got = 0;
    bool ok = true;
    KItem x;
    while (ok && next(n_got, x)) {
      int t = x.t0;
      for (int i = 0; i < x.n; ++i, ++g) {
        // column c of this quarter sees key row r where c >= r - shift
        const int shift = x.diag + 128 * t + 32 * quarter;
        if (++t == x.tiles) t = 0;
        const bool masked = p.causal && (warp & 3) * 32 + 31 > shift;
        const int slot = (int)(g % NROW);
        const float* nl = rowv + slot * 256 + 32 * quarter + col0;
        if (!warp_wait(bars + L::kRowFull + slot, (g / NROW) & 1, abort_flag, p.status) ||
            !warp_wait(bars + L::kSFull, g & 1, abort_flag, p.status)) { ok = false; break; }
        tc_fence_after_sync();
        // S is complete, and with it the dV issued before it: its dO tile is free
        if (warp == 4 && lane == 0 && g > 0) mbar_arrive(bars + L::kEmpty + (int)((2 * g - 1) % NST));
        // v[16 u + 4 i + 2 b + e]: key row0 + 16 u + 8 b, column 8 i + col0 + e
        uint32_t v[32];
        tmem_ld_16x256(t_lane + kKS, v, 0);
        tmem_ld_16x256(t_lane + kKS + kUpper, v, 16);
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
        const int under = row0 - col0 - shift;  // element (u, i, b, e) is masked where 8 i + e - 16 u - 8 b < under
        auto probs = [&](auto mk) {
          constexpr bool kMask = decltype(mk)::value;
          uint64_t ll[4];
#pragma unroll
          for (int i8 = 0; i8 < 4; ++i8) {
            const float2 l2 = *reinterpret_cast<const float2*>(nl + 8 * i8);
            ll[i8] = pk2(l2.x, l2.y);
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t pk[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int e = 16 * u + 2 * k;
              float a, b;
              upk2(ffma2(pk2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), cc, ll[k >> 1]), a, b);
              if (kMask) {
                const int at = 8 * (k >> 1) - 16 * u - 8 * (k & 1);
                if (at < under) a = -INFINITY;
                if (at + 1 < under) b = -INFINITY;
              }
              if (!kMask && (k & 7) < DENSE_BWD_POLY8) {
                upk2(exp2_fma2_any(a, b), a, b);
              } else {
                a = fast_exp2(a);
                b = fast_exp2(b);
              }
              v[e] = __float_as_uint(a);
              v[e + 1] = __float_as_uint(b);
              pk[k] = pack_bf16x2(a, b);
            }
            tmem_st_16x128(t_lane + kKS + u * kUpper, pk);
          }
        };
        if (masked) probs(std::true_type{});
        else probs(std::false_type{});
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + L::kPFull);
        if (!warp_wait(bars + L::kDPFull, g & 1, abort_flag, p.status)) { ok = false; break; }
        tc_fence_after_sync();
        uint64_t dd[4];
#pragma unroll
        for (int i8 = 0; i8 < 4; ++i8) {
          const float2 d2 = *reinterpret_cast<const float2*>(nl + 128 + 8 * i8);
          dd[i8] = pk2(d2.x, d2.y);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t dp[16], pk[8];
          tmem_ld_16x256(t_lane + kKDP + u * kUpper, dp, 0);
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
          if (masked) {
            // p = 0 there, but dP may be infinite
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (8 * (k >> 2) + (k & 1) - 16 * u - 8 * ((k >> 1) & 1) < under) dp[k] = 0u;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int e = 16 * u + 2 * k;
            float a, b;
            upk2(fmul2(fadd2(pk2(__uint_as_float(dp[2 * k]), __uint_as_float(dp[2 * k + 1])), dd[k >> 1]),
                       pk2(__uint_as_float(v[e]), __uint_as_float(v[e + 1]))), a, b);
            pk[k] = pack_bf16x2(a, b);
          }
          tmem_st_16x128(t_lane + kKDP + u * kUpper, pk);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bars + L::kDSFull);
          mbar_arrive(bars + L::kRowEmpty + slot);
        }
      }
    }
  } else {
    // ===================== results: one thread per key =====================
    const int row = (warp & 3) * 32 + lane;
    const uint32_t t_lane = tmem_base + (uint32_t((warp & 3) * 32) << 16);
    uint32_t n_item = 0, n_got = 0;
    KItem x;
    while (next(n_got, x)) {
      const bool real = row < x.keys;
      __nv_bfloat16* tk = p.dk + x.hk * p.dk_st.h + (long long)(x.key0 + row) * p.dk_st.s;
      __nv_bfloat16* tv = p.dv + x.hk * p.dv_st.h + (long long)(x.key0 + row) * p.dv_st.s;
      bool ok = true;
#pragma unroll 1
      for (int k = 0; ok && k < 2; ++k) {  // dV, then dK
        ok = warp_wait(bars + (k ? L::kDKFull : L::kDVFull), n_item & 1, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after_sync();
        __nv_bfloat16* to = k ? tk : tv;
        const float m = k ? p.scale : 1.f;
#pragma unroll 1
        for (int q0 = 0; q0 < D; q0 += 32) {
          uint32_t ov[32];
          tmem_ld32(t_lane + (k ? kKDK : kKDV) + q0, ov);
          if (q0 + 32 == D) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars + (k ? L::kDKEmpty : L::kDVEmpty));
          }
          if (!real) continue;
          if (p.parts > 1) {
            float* sum = part_row<D>(p, x, row) + (k ? 0 : (long long)p.Hkv * p.part_rows * D);
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(sum + q0 + e) = make_uint4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
            continue;
          }
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t o[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              o[q] = pack_bf16x2(__uint_as_float(ov[e + 2 * q]) * m, __uint_as_float(ov[e + 2 * q + 1]) * m);
            *reinterpret_cast<uint4*>(to + q0 + e) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      }
      if (!ok) break;
      ++n_item;
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

// ---------------------------------------------------------------------------
// the sum of the items that shared a key tile: eight elements a thread, parts in order
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(256) dense_dkv_join_kernel(const __grid_constant__ DenseBwdParams p) {
  const long long per = (long long)p.Hkv * p.part_rows * (D / 8);  // of one gradient
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= 2 * per) return;
  const bool is_v = i >= per;
  const long long j = is_v ? i - per : i;
  const int ch = (int)(j % (D / 8));
  const long long hr = j / (D / 8);
  const int row = (int)(hr % p.part_rows), h = (int)(hr / p.part_rows);
  float sum[8] = {};
#pragma unroll 4
  for (int k = 0; k < p.parts; ++k) {
    const float4* from = reinterpret_cast<const float4*>(p.part + k * (16 * per) + i * 8);
    const float4 a = from[0], b = from[1];
    sum[0] += a.x, sum[1] += a.y, sum[2] += a.z, sum[3] += a.w;
    sum[4] += b.x, sum[5] += b.y, sum[6] += b.z, sum[7] += b.w;
  }
  const float m = is_v ? 1.f : p.scale;
  uint32_t o[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) o[q] = pack_bf16x2(sum[2 * q] * m, sum[2 * q + 1] * m);
  const Strides3& st = is_v ? p.dv_st : p.dk_st;
  __nv_bfloat16* to = (is_v ? p.dv : p.dk) + h * st.h + (long long)(p.part_row0 + row) * st.s + 8 * ch;
  *reinterpret_cast<uint4*>(to) = make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace
}  // namespace dense

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int dkv_parts(const int4* seqs, int n, int Hq, int Hkv, bool causal) {
  const int sms = device_sm_count();
  long long items = 0;
  for (int i = 0; i < n; ++i) items += (seqs[i].w + 127LL) / 128 * Hkv;
  if (items == 0 || items >= 2 * sms) return 1;  // (this also bounds the partial sums' memory)
  // query tiles that the longest item, and all of them, walk over
  long long longest = 0, total = 0;
  for (int i = 0; i < n; ++i)
    for (long long key = 0; key < seqs[i].w; key += 128) {
      const long long skip = causal ? std::max(0LL, key - (seqs[i].w - seqs[i].y)) : 0;
      const long long tiles = (std::max(0LL, seqs[i].y - skip) + 127) / 128 * (Hq / Hkv);
      longest = std::max(longest, tiles);
      total += tiles * Hkv;
    }
  // Sharing evens the SMs out and costs a launch and the partial sums, about what
  // 11 tiles take: one sequence of 2000 rows, 8 heads over 1: 249 us in one part,
  // 77 in 16; 384 rows, 4 over 1 (12 tiles at most): 44 and 38; 2000 rows, 8 heads
  // over 8 (16 tiles at most, 7 on average per SM): 71 and 89.
  if (longest - total / sms < 11) return 1;
  // two items or more to an SM, four tiles or more to an item
  return (int)std::min(std::min(16LL, longest / 4), std::max(2LL, (2 * sms + items - 1) / items));
}

static size_t dkv_part_bytes(const int4* seqs, int n, int parts, int Hkv, int D) {
  const long long rows = seqs[n - 1].z + (long long)seqs[n - 1].w - seqs[0].z;
  return parts == 1 ? 0 : (size_t)parts * 2 * Hkv * rows * D * sizeof(float);
}

// delta, then the partial sums of one launch after the other
static size_t delta_bytes(int Hq, long long q_rows) {
  return ((size_t)Hq * q_rows * sizeof(float) + 255) & ~size_t(255);
}

size_t dense_bwd_workspace(const DenseBatch& b, int Hq, int Hkv, int D, long long q_rows, bool causal) {
  size_t most = 0;
  for (int i0 = 0; i0 < b.n; i0 += kDenseMaxSeqs) {
    int4 seqs[kDenseMaxSeqs];
    const int n = b.chunk(i0, seqs);
    most = std::max(most, dkv_part_bytes(seqs, n, dkv_parts(seqs, n, Hq, Hkv, causal), Hkv, D));
  }
  return delta_bytes(Hq, q_rows) + most;
}

template <int D>
static int launch_dense_bwd_t(DenseBwdParams p, const CUtensorMap* m, const int4* seqs, int n,
                              cudaStream_t stream) {
  static KernelReady ready_q, ready_k;
  auto kq = dense::dense_dq_kernel<D>;
  auto kk = dense::dense_dkv_kernel<D>;
  int rc = ready_q.check(reinterpret_cast<const void*>(kq), (int)dense::QLayout<D>::kAlloc);
  if (rc == VSA_OK)
    rc = ready_k.check(reinterpret_cast<const void*>(kk), (int)dense::KLayout<D>::kAlloc);
  if (rc != VSA_OK) return rc;
  int units[kDenseMaxSeqs], flat[kDenseMaxSeqs];
  DenseSeqs table;
  long long q_units = 0, k_units = 0;
  for (int i = 0; i < n; ++i) {
    q_units += (seqs[i].y + 127LL) / 128 * p.Hq;
    k_units += (seqs[i].w + 127LL) / 128 * p.Hkv;
    if ((seqs[i].y + 127LL) / 128 * p.group >= (1 << 27)) return VSA_ERR_UNSUPPORTED;
  }
  p.parts = dkv_parts(seqs, n, p.Hq, p.Hkv, p.causal != 0);
  p.part_row0 = seqs[0].z;
  p.part_rows = seqs[n - 1].z + seqs[n - 1].w - seqs[0].z;
  p.part = reinterpret_cast<float*>(reinterpret_cast<char*>(p.delta) + delta_bytes(p.Hq, p.lse_seq));
  if (q_units >= (1 << 30) || k_units >= (1 << 30)) return VSA_ERR_UNSUPPORTED;  // 32-bit item index
  if (q_units > 0) {
    for (int i = 0; i < n; ++i) {
      units[i] = (seqs[i].y + 127) / 128 * p.group;
      // behind cached keys the first rows, too, have many to see
      flat[i] = !p.causal || seqs[i].w > seqs[i].y ? seqs[i].w : 0;
    }
    fill_dense_seqs(&table, seqs, units, flat, n);
    kq<<<(unsigned)q_units, dense::kThreads, dense::QLayout<D>::kAlloc, stream>>>(
        m[0], m[1], m[2], m[3], m[4], p, table);
  }
  if (k_units > 0) {
    for (int i = 0; i < n; ++i) {
      units[i] = (seqs[i].w + 127) / 128;
      flat[i] = p.causal ? 0 : seqs[i].y;
    }
    fill_dense_seqs(&table, seqs, units, flat, n);
    kk<<<(unsigned)(k_units * p.parts), dense::kThreads, dense::KLayout<D>::kAlloc, stream>>>(
        m[0], m[1], m[2], m[3], p, table);
    if (p.parts > 1) {
      const long long chunks = 2LL * p.Hkv * p.part_rows * (D / 8);
      dense::dense_dkv_join_kernel<D><<<(unsigned)((chunks + 255) / 256), 256, 0, stream>>>(p);
    }
  }
  return cudaGetLastError() == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
}

int launch_dense_bwd(const DenseBwdParams& p_in, const DenseTensors& t, const void* out, Strides3 out_st,
                     const void* dout, Strides3 do_st, const DenseBatch& b, int D, cudaStream_t stream) {
  DenseBwdParams p = p_in;
  // without rows or keys no tile is loaded; the maps only have to be valid
  const bool rows = t.q_seq > 0, keys = t.kv_seq > 0;
  const void* any = rows ? t.q : t.k;
  const long long any_seq = rows ? t.q_seq : t.kv_seq;
  const int any_h = rows ? p.Hq : p.Hkv;
  const Strides3 any_st = rows ? t.q_st : t.k_st;
  CUtensorMap m[5];
  auto map = [&](CUtensorMap* to, TmaAxes* ax, bool have, const void* base, long long seq, int H, Strides3 st) {
    return have ? make_view_map_rows(to, ax, base, D, seq, H, 1, st, 128)
                : make_view_map_rows(to, ax, any, D, any_seq, any_h, 1, any_st, 128);
  };
  if (!map(&m[0], &p.q_ax, rows, t.q, t.q_seq, p.Hq, t.q_st) ||
      !map(&m[1], &p.k_ax, keys, t.k, t.kv_seq, p.Hkv, t.k_st) ||
      !map(&m[2], &p.v_ax, keys, t.v, t.kv_seq, p.Hkv, t.v_st) ||
      !map(&m[3], &p.do_ax, rows, dout, t.q_seq, p.Hq, do_st) ||
      !map(&m[4], &p.o_ax, rows, out, t.q_seq, p.Hq, out_st))
    return VSA_ERR_CUDA;
  p.item_us = std::max(item_microseconds(b, false, 1), item_microseconds(b, true, p.group));
  for (int i0 = 0; i0 < b.n; i0 += kDenseMaxSeqs) {
    int4 seqs[kDenseMaxSeqs];
    const int n = b.chunk(i0, seqs);
    const int rc = D == 128 ? launch_dense_bwd_t<128>(p, m, seqs, n, stream)
                            : launch_dense_bwd_t<64>(p, m, seqs, n, stream);
    if (rc != VSA_OK) return rc;
  }
  return VSA_OK;
}

}  // namespace vsa

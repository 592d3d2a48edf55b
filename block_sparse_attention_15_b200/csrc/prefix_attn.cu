// Attention of the newest tokens of a batch of requests over a prefix that all
// requests share, stored once, and over each request's own suffix: decoding.
//
// What it computes, for request b, token t of T and query head h (key head
// h / G), with len = suffix_lens[b]:
//   out = softmax(scale q . [k_prefix; k_suffix[b, 0 : len - T + 1 + t]]) . [v ...]
// (the new tokens' own keys are the last T of the suffix); a row that sees no
// key gives 0.
//
// How (sm_100a).  The rows of all requests that read a key head, B * G * T of
// them, are stacked into 128-row tiles against the prefix, so its keys come
// from HBM once; the G * T rows of one request are a (mostly empty) tile
// against its suffix.  Both are the forward kernel's products (S = Q K^T, P in
// TMEM, O += P V); a 128-row tile with few real rows wastes tensor cycles, not
// time: 1024 cycles per 64 KB of K and V are 2.5 times what HBM feeds an SM.
// Rows without a query are skipped by the softmax.
//
// Work split: all (key head, segment, key tile) triples form one line (a
// segment is a row block of the prefix, or a request's suffix), cut into equal
// pieces, one per CTA, whatever the lengths are (they are read on the device).
// A CTA's part of a segment leaves a partial result (normalised rows, log2
// sums) in the workspace; segment + CTA numbers it, as both only grow along the
// line.  A second kernel joins each row's partials.
// Within a CTA the two slots share the key tiles: with more than 128 rows each
// slot takes half of the rows, otherwise both have the same rows and take
// alternate key tiles, two chains of product, softmax, product in flight.
//
// Warp roles as in the forward kernel; Q rows are gathered by the softmax
// warps themselves (they come from many requests), under the K/V prefetch.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dense_attn.cuh"
#include "dense_launch.h"
#include "vsa.h"
#include "vsa_device.cuh"

namespace vsa {
namespace prefix {

using dense::issue_pv;
using dense::issue_s;

constexpr int kThreads = 512;
constexpr uint32_t kRegsProducer = 80, kRegsSoftmax = 184, kRegsEpilogue = 64;
constexpr uint32_t kLaunchRegs = 128;
static_assert(128u * (kRegsProducer + 2u * kRegsSoftmax + kRegsEpilogue) <= 512u * kLaunchRegs,
              "register split exceeds the launch's registers");
constexpr float kRefresh = 8.f;

template <int D>
struct Layout {
  static constexpr int DH = D / 64;
  static constexpr uint32_t kTile = 128u * D * 2u;
  static constexpr int NST = D == 128 ? 5 : 10;
  static constexpr uint32_t kQOff = 0;  // [2]
  static constexpr uint32_t kRingOff = kQOff + 2 * kTile;
  static constexpr uint32_t kInvLOff = kRingOff + NST * kTile;  // [2][128] f32
  static constexpr uint32_t kBarOff = kInvLOff + 2u * 128u * 4u;
  static constexpr int kQFull = 0, kFull = 2, kEmpty = kFull + NST, kPre = kEmpty + NST,
                       kSFull = kPre + NST, kPFull = kSFull + 2, kOFull = kPFull + 2,
                       kOEmpty = kOFull + 2, kLFull = kOEmpty + 2, kNumBars = kLFull + 2;
  static constexpr uint32_t kMiscOff = kBarOff + 8u * kNumBars;
  static constexpr uint32_t kBytes = kMiscOff + 16u;
  static constexpr uint32_t kAlloc = kBytes + 1024u;
  static_assert(kAlloc <= 227u * 1024u, "shared memory");
};

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 256;

// Real suffix keys of request b; a length outside [0, capacity] counts as 0.
__device__ __forceinline__ int suffix_len(const PrefixParams& p, int b) {
  const int n = p.lens[b];
  return n < 0 || n > p.suffix_cap ? 0 : n;
}

__device__ __forceinline__ int key_tiles(int keys) { return (keys + 127) >> 7; }

// The line of key tiles (see the header comment).  Whole-warp functions: every
// lane gets the same answer.
struct Line {
  int per_head;     // tiles of one key head
  long long total;  // tiles of all key heads
  int ctas;         // CTAs that share them: with fewer tiles than CTAs, the first ones take one each
};

// Tiles of the suffixes of requests [0, b_end).
__device__ __forceinline__ int suffix_tiles_before(const PrefixParams& p, int b_end, int lane) {
  int sum = 0;
  for (int b = lane; b < b_end; b += 32) sum += key_tiles(suffix_len(p, b));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum * p.sfx_blocks;
}

__device__ __forceinline__ Line make_line(const PrefixParams& p, int lane, int grid) {
  Line l;
  l.per_head = p.pfx_blocks * key_tiles(p.prefix_len) + suffix_tiles_before(p, p.B, lane);
  l.total = (long long)l.per_head * p.Hkv;
  l.ctas = l.total < grid ? (int)l.total : grid;
  return l;
}

// CTA whose piece of the line holds tile x.
__device__ __forceinline__ int cta_of(const Line& l, long long x) {
  return (int)(((x + 1) * l.ctas + l.total - 1) / l.total) - 1;
}

// One CTA's part of one segment.
struct Piece {
  int h;          // key head
  int b;          // request, -1: the prefix
  int blk;        // row block of 256
  int tile0, nt;  // key tiles
  int kv_len;     // keys of the segment
  int rows;       // rows of the block
  long long part; // partial-result number within its kind
};

// The CTA's pieces in order.
struct Walk {
  const PrefixParams& p;
  Line line;
  long long at, end;  // tiles [at, end) are still to do
  int h, b, blk, tile;  // where `at` lies (b = -1: the prefix)

  __device__ __forceinline__ Walk(const PrefixParams& pp, int lane) : p(pp) {
    line = make_line(p, lane, gridDim.x);
    const long long c = blockIdx.x;
    at = end = 0;
    if (c < line.ctas) {
      at = line.total * c / line.ctas;
      end = line.total * (c + 1) / line.ctas;
    }
    h = 0;
    b = -1;
    blk = tile = 0;
    if (at >= end) return;
    h = (int)(at / line.per_head);
    int r = (int)(at - (long long)h * line.per_head);
    const int tp = key_tiles(p.prefix_len);
    if (r < p.pfx_blocks * tp) {
      blk = r / tp;
      tile = r - blk * tp;
      return;
    }
    r -= p.pfx_blocks * tp;
    // the request whose suffix holds tile r: 32 requests at a time
    for (int b0 = 0;; b0 += 32) {
      const int mine = b0 + lane < p.B ? key_tiles(suffix_len(p, b0 + lane)) * p.sfx_blocks : 0;
      int sum = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      const int all = __shfl_sync(0xffffffffu, sum, 31);
      if (r >= all && b0 + 32 < p.B) {
        r -= all;
        continue;
      }
      const unsigned past = __ballot_sync(0xffffffffu, sum > r);
      const int i = past ? __ffs(past) - 1 : 31;
      r -= __shfl_sync(0xffffffffu, sum - mine, i);
      b = b0 + i;
      break;
    }
    const int tb = max(1, key_tiles(suffix_len(p, b)));
    blk = r / tb;
    tile = r - blk * tb;
  }

  __device__ __forceinline__ bool next(Piece& x) {
    if (at >= end) return false;
    // step over what holds no tile
    for (;;) {
      const int len = b < 0 ? p.prefix_len : suffix_len(p, b);
      const int blocks = b < 0 ? p.pfx_blocks : p.sfx_blocks;
      if (blk < blocks && tile < key_tiles(len)) {
        x.kv_len = len;
        break;
      }
      tile = 0;
      if (++blk < blocks && len > 0) continue;
      blk = 0;
      if (++b == p.B) {
        b = -1;
        if (++h >= p.Hkv) return false;  // not reached while at < end
      }
    }
    x.h = h;
    x.b = b;
    x.blk = blk;
    x.tile0 = tile;
    const long long left = end - at;
    const int here = key_tiles(x.kv_len) - tile;
    x.nt = left < here ? (int)left : here;
    const int rows = b < 0 ? p.B * p.rows_per_req : p.rows_per_req;
    x.rows = min(256, rows - 256 * blk);
    x.part = (b < 0 ? (long long)h * p.pfx_blocks + blk
                    : ((long long)h * p.B + b) * p.sfx_blocks + blk) + blockIdx.x;
    at += x.nt;
    tile += x.nt;
    return true;
  }
};

// Key tiles of a slot and which they are.
__device__ __forceinline__ bool split_rows(const Piece& x) { return x.rows > 128; }
__device__ __forceinline__ int slot_tiles(const Piece& x, int s) {
  return split_rows(x) ? x.nt : (x.nt + 1 - s) >> 1;
}
__device__ __forceinline__ int slot_tile(const Piece& x, int s, int j) {
  return split_rows(x) ? j : 2 * j + s;
}
// Real rows of a slot.
__device__ __forceinline__ int slot_rows(const Piece& x, int s) {
  return split_rows(x) ? min(128, x.rows - 128 * s) : x.rows;
}

// Row r of the piece's row block: request, head and token.
struct Row {
  int b, head, t;
};
__device__ __forceinline__ Row find_row(const PrefixParams& p, const Piece& x, int r) {
  int i = 256 * x.blk + r;
  Row o;
  o.b = x.b;
  if (x.b < 0) {
    o.b = i / p.rows_per_req;
    i -= o.b * p.rows_per_req;
  }
  const int g = i / p.T;
  o.head = x.h * p.group + g;
  o.t = i - g * p.T;
  return o;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_attn_kernel(const __grid_constant__ CUtensorMap tm_kp, const __grid_constant__ CUtensorMap tm_vp,
                       const __grid_constant__ CUtensorMap tm_ks, const __grid_constant__ CUtensorMap tm_vs,
                       const __grid_constant__ PrefixParams p) {
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

  if (tid == 0) {
    for (int i = 0; i < L::kNumBars; ++i) {
      const bool four = i < L::kFull || (i >= L::kPFull && i < L::kPFull + 2) || i >= L::kOEmpty;
      mbar_init(bars + i, four ? 4u : 1u);
    }
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_kp);
    tma_prefetch_desc(&tm_vp);
    tma_prefetch_desc(&tm_ks);
    tma_prefetch_desc(&tm_vs);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;

  if (warp < 4) {
    regs_dec<kRegsProducer>();
    if (warp == 0) {
      // ===================== K and V tiles =====================
      if (blockIdx.x == 0)
        for (int b = lane; b < p.B; b += 32)
          if (p.lens[b] < 0 || p.lens[b] > p.suffix_cap) set_status(p.status, VSA_ERR_INDEX_RANGE);
      const uint64_t pol_p = l2_policy_evict_last(), pol_s = l2_policy_evict_first();
      Walk walk(p, lane);
      Piece x;
      uint32_t g = 0;
      bool ok = true;
      while (ok && walk.next(x)) {
        if (lane == 0) {
          const bool own = x.b >= 0;
          const int b = own ? x.b : 0;
          for (int j = 0; ok && j < 2 * x.nt; ++j, ++g) {
            const int st = (int)(g % NST);
            const uint32_t u = g / NST;
            if (u >= 1) ok = mbar_wait(bars + L::kEmpty + st, (u - 1) & 1, abort_flag, p.status);
            if (!ok) break;
            const bool is_v = j & 1;
            const int key = 128 * (x.tile0 + (j >> 1));
            uint64_t* full = bars + (is_v && x.kv_len - key < 128 ? L::kPre : L::kFull) + st;
            uint8_t* dst = smem + L::kRingOff + st * L::kTile;
            const CUtensorMap* map = own ? (is_v ? &tm_vs : &tm_ks) : (is_v ? &tm_vp : &tm_kp);
            const TmaAxes ax = own ? (is_v ? p.vs_ax : p.ks_ax) : (is_v ? p.vp_ax : p.kp_ax);
            mbar_arrive_expect_tx(full, L::kTile);
#pragma unroll
            for (int dh = 0; dh < L::DH; ++dh)
              dense::load_rows(dst + dh * 16384, map, ax, full, dh * 64, key, x.h, b, own ? pol_s : pol_p);
          }
        }
        g = __shfl_sync(0xffffffffu, g, 0);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      }
      if (lane == 0)
        for (uint32_t t = (g > (uint32_t)NST ? g - NST : 0u); ok && t < g; ++t)
          ok = mbar_wait(bars + L::kEmpty + (int)(t % NST), (t / NST) & 1, abort_flag, p.status);
      __syncwarp();
    } else if (warp == 2) {
      // ============ zero V rows past a segment's keys (what a cache holds there) ============
      Walk walk(p, lane);
      Piece x;
      uint32_t g = 0, pre = 0;
      while (walk.next(x)) {
        g += 2 * x.nt;
        const int len = x.kv_len - 128 * (x.tile0 + x.nt - 1);
        if (len >= 128) continue;
        const int st = (int)((g - 1) % NST);
        if (!warp_wait(bars + L::kPre + st, (pre >> st) & 1, abort_flag, p.status)) break;
        pre ^= 1u << st;
        dense::zero_rows<128>(smem + L::kRingOff + st * L::kTile, L::DH, len, (len + 15) & ~15, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + L::kFull + st);
      }
    } else if (warp == 1) {
      // ===================== MMA issue =====================
      uint32_t cs[2] = {0, 0};  // pieces of the slot that have started
      uint32_t gs[2] = {0, 0};  // key tiles of the slot whose P has been consumed
      uint32_t g = 0;
      bool ok = true;
      auto do_s = [&](const Piece& x, int s, int j, uint32_t g_piece) {
        const int tile = slot_tile(x, s, j);
        const uint32_t gk = g_piece + 2 * tile;
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
          if (s == 1 || !split_rows(x)) umma_commit(bars + L::kEmpty + st);
        }
        __syncwarp();
      };
      Walk walk(p, lane);
      Piece x;
      while (ok && walk.next(x)) {
        const int n0 = slot_tiles(x, 0), n1 = slot_tiles(x, 1);
        do_s(x, 0, 0, g);
        if (ok && n1 > 0) do_s(x, 1, 0, g);
        for (int j = 0; ok && j < n0; ++j) {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int ns = s ? n1 : n0;
            if (!ok || j >= ns) continue;
            const int tile = slot_tile(x, s, j);
            const uint32_t gv = g + 2 * tile + 1;
            const int st = (int)(gv % NST);
            if (j == 0 && cs[s] >= 2 &&
                !warp_wait(bars + L::kOEmpty + s, (cs[s] - 2) & 1, abort_flag, p.status)) { ok = false; continue; }
            if (!warp_wait(bars + L::kFull + st, (gv / NST) & 1, abort_flag, p.status)) { ok = false; continue; }
            if (!warp_wait(bars + L::kPFull + s, gs[s] & 1, abort_flag, p.status)) { ok = false; continue; }
            ++gs[s];
            tc_fence_after_sync();
            if (elect_one()) {
              const int keys = x.kv_len - 128 * (x.tile0 + tile);
              issue_pv<D>(tmem_base + kTmemO + D * s, tmem_base + 128u * s,
                          sbase + L::kRingOff + st * L::kTile, keys >= 128 ? 8 : (keys + 15) >> 4, j > 0);
              if (s == 1 || !split_rows(x)) umma_commit(bars + L::kEmpty + st);
              if (j == ns - 1) umma_commit(bars + L::kOFull + s);
            }
            __syncwarp();
            if (j + 1 < ns) do_s(x, s, j + 1, g);
          }
        }
        g += 2 * x.nt;
      }
    }
  } else if (warp < 12) {
    regs_inc<kRegsSoftmax>();
    // ===================== Q gather and softmax: one thread per row =====================
    const int s = (warp - 4) >> 2;
    const int wq = warp & 3;
    const int row = wq * 32 + lane;
    const uint32_t t_s = tmem_base + (uint32_t(wq * 32) << 16) + 128u * s;
    const uint32_t t_o = tmem_base + (uint32_t(wq * 32) << 16) + kTmemO + D * s;
    const float c = p.scale_log2;
    const uint64_t cc = pk2(c, c);
    uint8_t* qt = smem + L::kQOff + s * L::kTile;
    uint32_t g = 0, n = 0;
    bool ok = true;
    Walk walk(p, lane);
    Piece x;
    while (ok && walk.next(x)) {
      const int nt = slot_tiles(x, s);
      const int rows = slot_rows(x, s);
      const int first = split_rows(x) ? 128 * s : 0;  // the slot's first row in the block
      float* lse_out = (x.b < 0 ? p.part_lse_p + x.part * (2 * p.pfx_rows) + s * p.pfx_rows
                                : p.part_lse_s + x.part * (2 * p.sfx_rows) + s * p.sfx_rows);
      if (nt == 0) {
        // a piece of one key tile leaves slot 1 nothing
        if (row < rows) lse_out[row] = -INFINITY;
        continue;
      }
      // The slot's score products up to here are complete (their results were
      // waited for), so its Q tile may be overwritten.  Each warp fetches its
      // own 32 rows: 16-byte chunks, consecutive lanes along a row, into the
      // 128-byte swizzle.  Rows past the block keep what the tile held; only
      // their own (unused) results depend on it.
      constexpr int CH = D / 8;
      const int my_rows = min(32, max(0, rows - 32 * wq));
#pragma unroll 8
      for (int i = lane; i < my_rows * CH; i += 32) {
        const int r = 32 * wq + i / CH, ch = i % CH;
        const Row o = find_row(p, x, first + r);
        const uint4 v = *reinterpret_cast<const uint4*>(p.q + o.b * p.q_st.b + o.head * p.q_st.h +
                                                        (long long)o.t * p.q_st.s + ch * 8);
        *reinterpret_cast<uint4*>(qt + (ch >> 3) * 16384 + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = v;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + L::kQFull + s);
      const bool any = 32 * wq < rows;  // this warp has rows
      int limit = x.kv_len;             // keys the row sees
      if (x.b >= 0 && row < rows) limit = x.kv_len - p.T + 1 + find_row(p, x, first + row).t;
      float m = -INFINITY;
      uint64_t l2 = pk2(0.f, 0.f);
      for (int j = 0; j < nt; ++j, ++g) {
        if (!warp_wait(bars + L::kSFull + s, g & 1, abort_flag, p.status)) { ok = false; break; }
        tc_fence_after_sync();
        if (any) {
          uint32_t v[128];
#pragma unroll
          for (int q = 0; q < 8; ++q) VSA_TMEM_LD16(t_s + 16u * q, v, 16 * q);
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
          const int rem = limit - 128 * (x.tile0 + slot_tile(x, s, j));
          const bool masked = __any_sync(0xffffffffu, rem < 128);
          if (masked) {
#pragma unroll
            for (int q = 0; q < 128; ++q)
              if (q >= rem) v[q] = __float_as_uint(-INFINITY);
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int q = 0; q < 128; q += 8) {
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
              // PV(j - 1) is complete: the thread that issued S(j) issued it before
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
          const float ref = (m == -INFINITY) ? 0.f : -m;
          const uint64_t nm2 = pk2(ref, ref);
#pragma unroll
          for (int q0 = 0; q0 < 64; q0 += 16) {
            uint32_t pk[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const int e = 2 * (q0 + q);
              float a, b;
              upk2(ffma2(pk2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), cc, nm2), a, b);
              const float p0 = fast_exp2(a), p1 = fast_exp2(b);
              l2 = fadd2(l2, pk2(p0, p1));
              pk[q] = pack_bf16x2(p0, p1);
            }
            VSA_TMEM_ST16(t_s + q0, pk, 0);
          }
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + L::kPFull + s);
      }
      if (!ok) break;
      if (n >= 1 && !warp_wait(bars + L::kOEmpty + s, (n - 1) & 1, abort_flag, p.status)) { ok = false; break; }
      ++n;
      float la, lb;
      upk2(l2, la, lb);
      const float l = la + lb;
      inv_l[s * 128 + row] = l == 0.f ? 0.f : 1.f / l;
      if (row < rows) lse_out[row] = l == 0.f ? -INFINITY : m + __log2f(l);
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + L::kLFull + s);
    }
  } else {
    regs_dec<kRegsEpilogue>();
    // ===================== epilogue: partial rows in fp32 =====================
    const int wq = warp - 12;
    const int row = wq * 32 + lane;
    const uint32_t t_lane = tmem_base + (uint32_t(wq * 32) << 16) + kTmemO;
    uint32_t cs[2] = {0, 0};
    bool ok = true;
    Walk walk(p, lane);
    Piece x;
    while (ok && walk.next(x)) {
#pragma unroll 1
      for (int s = 0; s < 2; ++s) {
        if (slot_tiles(x, s) == 0) continue;
        const uint32_t ph = cs[s] & 1;
        ++cs[s];
        if (!warp_wait(bars + L::kLFull + s, ph, abort_flag, p.status) ||
            !warp_wait(bars + L::kOFull + s, ph, abort_flag, p.status)) { ok = false; break; }
        tc_fence_after_sync();
        const int rows = slot_rows(x, s);
        if (32 * wq < rows) {
          const float il = inv_l[s * 128 + row];
          float* o = (x.b < 0 ? p.part_p + (x.part * (2 * p.pfx_rows) + s * p.pfx_rows + row) * D
                              : p.part_s + (x.part * (2 * p.sfx_rows) + s * p.sfx_rows + row) * D);
#pragma unroll
          for (int q0 = 0; q0 < D; q0 += 32) {
            uint32_t ov[32];
            tmem_ld32(t_lane + D * s + q0, ov);
            if (row < rows) {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4*>(o + q0 + e) =
                    make_float4(__uint_as_float(ov[e]) * il, __uint_as_float(ov[e + 1]) * il,
                                __uint_as_float(ov[e + 2]) * il, __uint_as_float(ov[e + 3]) * il);
            }
          }
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + L::kOEmpty + s);
      }
    }
  }

  dense::settle_after_abort(abort_flag);
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

// Joins a row's partials: weights 2^(lse_i - max), fp32.  One block per row,
// its warps taking partials in turn.
constexpr int kJoinWarps = 4;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps)
    prefix_join_kernel(const __grid_constant__ PrefixParams p, int grid) {
  constexpr int E = D / 32;  // elements per lane
  __shared__ float sm_m[kJoinWarps], sm_l[kJoinWarps];
  __shared__ float sm_o[kJoinWarps][D];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int row = blockIdx.x % p.rows_per_req;  // (head of the group, token)
  const int bh = blockIdx.x / p.rows_per_req;
  const int h = bh % p.Hkv, b = bh / p.Hkv;
  const Line line = make_line(p, lane, grid);
  float m = -INFINITY, l = 0.f, o[E] = {};
  // partials [first, first + count), `copies` rows each `pitch` apart
  auto take = [&](const float* part, const float* lse, long long first, int count, int rows, int slot0,
                  int copies, int r) {
    for (int i = warp; i < count * copies; i += kJoinWarps) {
      const long long at = (first + i / copies) * (2 * rows) + (slot0 + i % copies) * rows + r;
      const float x = lse[at];
      if (x == -INFINITY) continue;
      const float nm = fmaxf(m, x);
      const float a = fast_exp2(m - nm), w = fast_exp2(x - nm);
      m = nm;
      l = l * a + w;
      const float* src = part + at * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * a + w * src[e];
    }
  };
  const int tp = key_tiles(p.prefix_len);
  if (tp > 0) {
    const int gr = b * p.rows_per_req + row, blk = gr >> 8, r = gr & 255;
    const bool split = min(256, p.B * p.rows_per_req - 256 * blk) > 128;
    const long long t0 = (long long)h * line.per_head + (long long)blk * tp;
    const int c0 = cta_of(line, t0), c1 = cta_of(line, t0 + tp - 1);
    take(p.part_p, p.part_lse_p, (long long)h * p.pfx_blocks + blk + c0, c1 - c0 + 1, p.pfx_rows,
         split ? r >> 7 : 0, split ? 1 : 2, split ? r & 127 : r);
  }
  const int tb = key_tiles(suffix_len(p, b));
  if (tb > 0) {
    const int blk = row >> 8, r = row & 255;
    const bool split = min(256, p.rows_per_req - 256 * blk) > 128;
    const long long t0 = (long long)h * line.per_head + (long long)p.pfx_blocks * tp +
                         suffix_tiles_before(p, b, lane) + (long long)blk * tb;
    const int c0 = cta_of(line, t0), c1 = cta_of(line, t0 + tb - 1);
    take(p.part_s, p.part_lse_s, ((long long)h * p.B + b) * p.sfx_blocks + blk + c0, c1 - c0 + 1,
         p.sfx_rows, split ? r >> 7 : 0, split ? 1 : 2, split ? r & 127 : r);
  }
  if (lane == 0) {
    sm_m[warp] = m;
    sm_l[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sm_o[warp][lane * E + e] = o[e];
  __syncthreads();
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) top = fmaxf(top, sm_m[i]);
  float sum = 0.f, w[kJoinWarps];
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) {
    w[i] = sm_m[i] == -INFINITY ? 0.f : fast_exp2(sm_m[i] - top);
    sum += sm_l[i] * w[i];
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int g = row / p.T, t = row - g * p.T;
  const int head = h * p.group + g;
  __nv_bfloat16* out = p.out + b * p.out_st.b + head * p.out_st.h + (long long)t * p.out_st.s;
  for (int d = threadIdx.x; d < D; d += 32 * kJoinWarps) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kJoinWarps; ++i) v += w[i] * sm_o[i][d];
    out[d] = __float2bfloat16(v * inv);
  }
  if (p.lse && threadIdx.x == 0)
    p.lse[((long long)b * p.Hq + head) * p.T + t] =
        sum == 0.f ? -INFINITY : (top + __log2f(sum)) * 0.69314718055994531f;
}

}  // namespace prefix

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
void prefix_shape(PrefixParams* p) {
  p->group = p->Hq / p->Hkv;
  p->rows_per_req = p->group * p->T;
  const int all = p->B * p->rows_per_req;
  p->pfx_blocks = (all + 255) / 256;
  p->sfx_blocks = (p->rows_per_req + 255) / 256;
  p->pfx_rows = all < 128 ? all : 128;
  p->sfx_rows = p->rows_per_req < 128 ? p->rows_per_req : 128;
}

// Partial results of each kind: segments + CTAs, two slots of rows each.
static size_t parts_of(long long segments, int rows) {
  return (size_t)(segments + kPrefixGrid) * 2 * rows;
}
static size_t a256(size_t x) { return (x + 255) & ~size_t(255); }

size_t prefix_workspace(PrefixParams* p, int D, void* base) {
  prefix_shape(p);
  const bool pfx = p->prefix_len > 0, sfx = p->suffix_cap > 0;
  const size_t np = pfx ? parts_of((long long)p->Hkv * p->pfx_blocks, p->pfx_rows) : 0;
  const size_t ns = sfx ? parts_of((long long)p->Hkv * p->B * p->sfx_blocks, p->sfx_rows) : 0;
  char* at = static_cast<char*>(base);
  size_t off = 0;
  auto take = [&](size_t floats) {
    float* r = reinterpret_cast<float*>(at + off);
    off += a256(floats * sizeof(float));
    return r;
  };
  p->part_p = take(np * D);
  p->part_s = take(ns * D);
  p->part_lse_p = take(np);
  p->part_lse_s = take(ns);
  return off;
}

template <int D>
static int launch_prefix_t(const PrefixParams& p, const CUtensorMap* m, cudaStream_t stream) {
  using L = prefix::Layout<D>;
  auto kern = prefix::prefix_attn_kernel<D>;
  static KernelReady ready;
  const int rc = ready.check(reinterpret_cast<const void*>(kern), (int)prefix::kLaunchRegs, (int)L::kAlloc);
  if (rc != VSA_OK) return rc;
  // at most one CTA per key tile there can be
  const long long cap = (long long)p.Hkv * ((long long)p.pfx_blocks * ((p.prefix_len + 127LL) / 128) +
                                            (long long)p.B * p.sfx_blocks * ((p.suffix_cap + 127LL) / 128));
  const int grid = cap < kPrefixGrid ? (int)(cap > 0 ? cap : 1) : kPrefixGrid;
  kern<<<grid, prefix::kThreads, L::kAlloc, stream>>>(m[0], m[1], m[2], m[3], p);
  prefix::prefix_join_kernel<D><<<(unsigned)(p.B * p.Hkv * p.rows_per_req), 32 * prefix::kJoinWarps, 0, stream>>>(p, grid);
  return cudaGetLastError() == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
}

int launch_prefix(const PrefixParams& p_in, const PrefixTensors& t, int D, cudaStream_t stream) {
  PrefixParams p = p_in;
  CUtensorMap m[4];
  const bool pfx = p.prefix_len > 0, sfx = p.suffix_cap > 0;
  // a part that is empty loads nothing; its map only has to be valid
  if (pfx && (!make_view_map_rows(&m[0], &p.kp_ax, t.k_prefix, D, p.prefix_len, p.Hkv, 1, t.kp_st, 128) ||
              !make_view_map_rows(&m[1], &p.vp_ax, t.v_prefix, D, p.prefix_len, p.Hkv, 1, t.vp_st, 128)))
    return VSA_ERR_CUDA;
  if (sfx && (!make_view_map_rows(&m[2], &p.ks_ax, t.k_suffix, D, p.suffix_cap, p.Hkv, p.B, t.ks_st, 128) ||
              !make_view_map_rows(&m[3], &p.vs_ax, t.v_suffix, D, p.suffix_cap, p.Hkv, p.B, t.vs_st, 128)))
    return VSA_ERR_CUDA;
  if (!pfx && !sfx) {
    TmaAxes ax;
    for (int i = 0; i < 4; ++i)
      if (!make_view_map_rows(&m[i], &ax, p.q, D, p.T, p.Hq, p.B, p.q_st, 128)) return VSA_ERR_CUDA;
  } else if (!pfx) {
    m[0] = m[2], m[1] = m[3], p.kp_ax = p.ks_ax, p.vp_ax = p.vs_ax;
  } else if (!sfx) {
    m[2] = m[0], m[3] = m[1], p.ks_ax = p.kp_ax, p.vs_ax = p.vp_ax;
  }
  return D == 128 ? launch_prefix_t<128>(p, m, stream) : launch_prefix_t<64>(p, m, stream);
}

}  // namespace vsa

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
// them, are stacked into row blocks of 256 against the prefix, so its keys come
// from HBM once (and from L2 for further blocks); the G * T rows of one request
// are a (mostly empty) block against its suffix.  Both are the forward kernel's
// products (S = Q K^T, P in TMEM, O += P V); a 128-row tile with few real rows
// wastes tensor cycles, not time: the two products take 1460 cycles per 64 KB
// of K and V, for which an SM's share of HBM takes 2600.
//
// Work split: all (key head, segment, key tile) triples form one line (a
// segment is a row block of the prefix, or a request's suffix), cut into equal
// pieces, one per CTA, whatever the lengths are (they are read on the device).
// A CTA's part of a segment leaves a partial result (normalised rows, log2
// sums) in the workspace; segment + CTA numbers it, as both only grow along the
// line.  A second kernel joins each row's partials.  Where requests are many, a
// kernel before them adds up their key tiles.
// Within a CTA the two slots share the key tiles: with more than 128 rows each
// slot takes half of the rows, otherwise both have the same rows and take
// alternate key tiles, two chains of product, softmax, product in flight, and
// their results are joined on the way out.
//
// 512 threads: warp 0 loads K and V tiles, warp 1 (one thread) issues products,
// warp 2 zeroes what a segment's last V tile holds past its keys, warp 3 walks
// the line, warps 4-7 and 8-11 are the slots' softmax (one thread per row, or four
// where there are few; warps without rows pass), warps 12-15 gather the next piece's Q rows and write the
// last one's results.  Loops are kept short: the first pass through each line of
// code costs an instruction fetch that waits behind the K/V stream (a softmax
// unrolled over its 128 columns spent 25 us of a call on that).
//
// Measured at D = 128: 24 requests of 9216 keys at most, 56 heads over 8, no
// prefix: 84-87 us, 5.2-5.4 TB/s; 64 requests behind 15488 shared keys, 40 heads
// over 8: 93-99 us, 3.5 TB/s (a tile of the prefix takes 4600 cycles for its 256
// rows, one of a suffix 2300: every SM is busy, fewer than half of the time with a
// stream); 16 requests of 5 tokens: 38-40 us.
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
namespace prefix {

using dense::slim::mbar_wait;
using dense::slim::warp_wait;

constexpr int kThreads = 512;
constexpr float kRefresh = 8.f;

// One CTA's part of one segment.
struct Piece {
  int h;          // key head
  int b;          // request, -1: the prefix
  int blk;        // row block of 256
  int tile0, n;   // key tiles
  int kv_len;     // keys of the segment
  int rows;       // rows of the block
  int turn;       // slot that takes the first tile (of a block of up to 128 rows)
  long long part; // partial-result number within its kind
};

using PieceRing = dense::ItemRing<Piece, 4>;

template <int D>
struct Layout {
  static constexpr int DH = D / 64;
  static constexpr uint32_t kTile = 128u * D * 2u;
  static constexpr int NST = D == 128 ? 5 : 10;
  static constexpr uint32_t kQOff = 0;  // [2]
  static constexpr uint32_t kRingOff = kQOff + 2 * kTile;
  static constexpr uint32_t kMLOff = kRingOff + NST * kTile;  // [2 slots][m, l][128] f32
  static constexpr uint32_t kItemOff = kMLOff + 2048u;
  static constexpr uint32_t kBarOff = kItemOff + (uint32_t)sizeof(PieceRing);
  // kQFull and kQFree alternate between pieces: one piece may be ahead of a waiter
  static constexpr int kQFull = 0, kQFree = 2, kFull = 4, kEmpty = kFull + NST, kPre = kEmpty + NST,
                       kSFull = kPre + NST, kPFull = kSFull + 2, kOFull = kPFull + 2,
                       kOEmpty = kOFull + 2, kLFull = kOEmpty + 2, kItFull = kLFull + 2,
                       kItEmpty = kItFull + PieceRing::kSlots, kNumBars = kItEmpty + PieceRing::kSlots;
  static constexpr uint32_t kMiscOff = kBarOff + 8u * kNumBars;
  static constexpr uint32_t kAlloc = kMiscOff + 16u;
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

// The line of key tiles (see the header comment), measured in units: a tile of a
// block of more than 128 rows costs both slots a pass (4600 cycles against 2300
// measured) and counts 2, others 1.  A tile belongs to the CTA that holds its
// first unit.  With fewer than two units to a CTA every tile counts 1: a CTA
// must not fall between the two units of a tile, where it would leave no partial
// result.  Whole-warp functions: every lane gets the same answer.
struct Line {
  int heavy;       // units of a tile of a block of more than 128 rows
  int pfx, sfx;    // units of one key tile over all row blocks of a prefix / suffix segment
  int per_head;    // units of one key head
  int each, more;  // a CTA has `each` units, the first `more` CTAs one more
};

// Sum of the key tiles of requests [0, b_end).
__device__ __forceinline__ int suffix_tiles_before(const PrefixParams& p, int b_end, int lane) {
  if (p.tiles_before) return p.tiles_before[b_end];
  int sum = 0;
  for (int b = lane; b < b_end; b += 32) sum += key_tiles(suffix_len(p, b));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// Units of a tile of row block `blk` of a segment of `rows` rows, and of a tile
// over all its blocks.
__device__ __forceinline__ int tile_units(const Line& l, int rows, int blk) {
  return rows - 256 * blk > 128 ? l.heavy : 1;
}
__device__ __forceinline__ int all_units(const Line& l, int rows, int blocks) {
  return (blocks - 1) * l.heavy + tile_units(l, rows, blocks - 1);
}

__device__ __forceinline__ Line make_line(const PrefixParams& p, int lane, int grid) {
  Line l;
  const int tp = key_tiles(p.prefix_len), ts = suffix_tiles_before(p, p.B, lane);
  int total = 0;
#pragma unroll 1
  for (l.heavy = 2;; l.heavy = 1) {
    l.pfx = all_units(l, p.B * p.rows_per_req, p.pfx_blocks);
    l.sfx = all_units(l, p.rows_per_req, p.sfx_blocks);
    l.per_head = l.pfx * tp + l.sfx * ts;
    total = l.per_head * p.Hkv;
    if (l.heavy == 1 || total >= 2 * grid) break;
  }
  l.each = total / grid;
  l.more = total - l.each * grid;
  return l;
}

// CTA whose piece of the line holds unit x.
__device__ __forceinline__ int cta_of(const Line& l, int x) {
  const int first = l.more * (l.each + 1);
  return x < first ? x / (l.each + 1) : l.more + (x - first) / l.each;
}

// The CTA's pieces in order.
struct Walk {
  const PrefixParams& p;
  Line line;
  int at, end;          // the next tile's first unit; the CTA's units end here
  int h, b, blk, tile;  // the next tile (b = -1: the prefix)
  int turn;             // slot whose turn it is

  // (only the warp that walks looks anything up)
  __device__ __forceinline__ Walk(const PrefixParams& pp, int lane, bool mine) : p(pp) {
    at = end = h = blk = tile = turn = 0;
    b = -1;
    if (!mine) return;
    line = make_line(p, lane, gridDim.x);
    const int c = blockIdx.x;
    at = line.each * c + min(c, line.more);
    end = at + line.each + (c < line.more ? 1 : 0);
    if (at >= end) return;
    h = at / line.per_head;
    int r = at - h * line.per_head;
    int tiles = key_tiles(p.prefix_len), rows = p.B * p.rows_per_req, blocks = p.pfx_blocks;
    if (r >= line.pfx * tiles) {
      r -= line.pfx * tiles;
      // the request whose suffix holds unit r
      if (p.tiles_before) {
        // the last request with no more than r units before it
        int lo = 0, hi = p.B - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (p.tiles_before[mid] * line.sfx <= r) lo = mid;
          else hi = mid - 1;
        }
        b = lo;
        r -= p.tiles_before[b] * line.sfx;
      } else {
        // 32 requests at a time
        for (int b0 = 0;; b0 += 32) {
          const int mine_u = b0 + lane < p.B ? key_tiles(suffix_len(p, b0 + lane)) * line.sfx : 0;
          int sum = mine_u;
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
          r -= __shfl_sync(0xffffffffu, sum - mine_u, i);
          b = b0 + i;
          break;
        }
      }
      tiles = max(1, key_tiles(suffix_len(p, b)));
      rows = p.rows_per_req;
      blocks = p.sfx_blocks;
    }
    blk = min(r / (line.heavy * tiles), blocks - 1);
    r -= blk * line.heavy * tiles;
    const int w = tile_units(line, rows, blk);
    tile = (r + w - 1) / w;  // a tile that began before `at` is the previous CTA's
    at += tile * w - r;
  }

  __device__ __forceinline__ bool next(Piece& x) {
    if (at >= end) return false;
    // step over what holds no (further) tile
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
    const int rows = b < 0 ? p.B * p.rows_per_req : p.rows_per_req;
    const int w = tile_units(line, rows, blk);
    x.h = h;
    x.b = b;
    x.blk = blk;
    x.tile0 = tile;
    x.n = min((end - at + w - 1) / w, key_tiles(x.kv_len) - tile);
    x.rows = min(256, rows - 256 * blk);
    x.part = (b < 0 ? (long long)h * p.pfx_blocks + blk
                    : ((long long)h * p.B + b) * p.sfx_blocks + blk) + blockIdx.x;
    // short pieces take turns, so that one slot's product, softmax, product
    // runs under the other's
    x.turn = x.rows > 128 ? 0 : turn;
    turn ^= x.n & 1;
    at += x.n * w;
    tile += x.n;
    return true;
  }
};

// Key tiles of a slot and which they are.
__device__ __forceinline__ bool split_rows(const Piece& x) { return x.rows > 128; }
__device__ __forceinline__ int slot_tiles(const Piece& x, int s) {
  return split_rows(x) ? x.n : (x.n + 1 - (s ^ x.turn)) >> 1;
}
__device__ __forceinline__ int slot_tile(const Piece& x, int s, int j) {
  return split_rows(x) ? j : 2 * j + (s ^ x.turn);
}
// Place of K and V of tile t among a piece's 2 n ring tiles: in the order of the
// products that read them.  Where the slots alternate that is S(0) S(1) PV(0) S(2)
// PV(1) ..: loaded tile by tile, a K would wait for the stage of a V that is read
// one product later (24 requests of 9216 keys: 89 us, in this order 85).
__device__ __forceinline__ int place_k(const Piece& x, int t) { return split_rows(x) ? 2 * t : max(0, 2 * t - 1); }
__device__ __forceinline__ int place_v(const Piece& x, int t) {
  return split_rows(x) ? 2 * t + 1 : min(2 * t + 2, 2 * x.n - 1);
}
// Real rows of a slot.
__device__ __forceinline__ int slot_rows(const Piece& x, int s) {
  return split_rows(x) ? min(128, x.rows - 128 * s) : x.rows;
}

// Brings the lanes of a warp together again: lanes that a wait has suspended wake
// one by one, and may go on one by one, shuffles and all, until an instruction
// that the warp issues as one (256 rows of Q gathered: 20000 cycles without this,
// 3000 with it).  Barriers 1 to 15 are the warps' own.
__device__ __forceinline__ void converge(int warp) {
  asm volatile("barrier.sync.aligned %0, 32;" ::"r"(warp) : "memory");
}

// Rows a softmax warp has, as a power of two.  A tile of few rows spreads them
// over the four warps (row i in TMEM lane 32 (i >> shift) + its low bits), four
// lanes to a row: such tiles come as fast as the chain of product, softmax,
// product lets them, and one thread to a row takes 2400 cycles for its 128
// columns, four take 1350 (24 requests of 9216 keys: 91 us, 89).
__device__ __forceinline__ int row_shift(const Piece& x) { return x.rows <= 32 ? 3 : 5; }

// The products, out of line: they are issued from several places.
template <int D>
static __device__ __noinline__ void s_product(uint32_t tmem_d, uint32_t q_base, uint32_t k_base) {
  dense::issue_s<D>(tmem_d, q_base, k_base);
}
template <int D>
static __device__ __noinline__ void pv_product(uint32_t tmem_o, uint32_t tmem_p, uint32_t v_base, int steps,
                                               bool accumulate) {
  dense::issue_pv<D>(tmem_o, tmem_p, v_base, steps, accumulate);
}

// Rows [r0, r_end) of a partial result, up to 32 in this warp's TMEM lanes: O (or both slots' O, D columns apart)
// from TMEM times the row's weight, which lane i has for row r0 + i.  Four
// lanes write 64 bytes of a row.
template <int D>
static __device__ __noinline__ void write_part(float* o, int r0, int r_end, int lane, uint32_t t_o, bool both,
                                           float w0, float w1) {
#pragma unroll 1
  for (int u = 0; u < 2; ++u) {
    if (r0 + 16 * u >= r_end) break;
    float a0[2], a1[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      a0[b] = __shfl_sync(0xffffffffu, w0, 16 * u + 8 * b + lane / 4);
      a1[b] = __shfl_sync(0xffffffffu, w1, 16 * u + 8 * b + lane / 4);
    }
    const uint32_t t_u = t_o + ((uint32_t)(16 * u) << 16);
#pragma unroll 1
    for (int q0 = 0; q0 < D; q0 += 32) {
      uint32_t va[16], vb[16];
      dense::tmem_ld_16x256(t_u + q0, va, 0);
      if (both) dense::tmem_ld_16x256(t_u + D + q0, vb, 0);
      asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        float f = __uint_as_float(va[k]) * a0[(k >> 1) & 1];
        if (both) f = fmaf(__uint_as_float(vb[k]), a1[(k >> 1) & 1], f);
        va[k] = __float_as_uint(f);
      }
      // pairs of lanes exchange halves of two column groups: 16 bytes each
      const bool odd = lane & 1;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int b = k & 1, lo = 8 * (k >> 1) + 2 * b, hi = lo + 4;  // registers of groups 2 (k / 2), + 1
        const int r = r0 + 16 * u + 8 * b + lane / 4;
        const uint32_t sx = odd ? va[lo] : va[hi], sy = odd ? va[lo + 1] : va[hi + 1];
        const uint32_t rx = __shfl_xor_sync(0xffffffffu, sx, 1), ry = __shfl_xor_sync(0xffffffffu, sy, 1);
        const uint4 f = odd ? make_uint4(rx, ry, va[hi], va[hi + 1]) : make_uint4(va[lo], va[lo + 1], rx, ry);
        if (r < r_end)
          *reinterpret_cast<uint4*>(o + (long long)r * D + q0 + 16 * (k >> 1) + (odd ? 8 : 0) + 2 * (lane & 2)) = f;
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_attn_kernel(const __grid_constant__ CUtensorMap tm_kp, const __grid_constant__ CUtensorMap tm_vp,
                       const __grid_constant__ CUtensorMap tm_ks, const __grid_constant__ CUtensorMap tm_vs,
                       const __grid_constant__ PrefixParams p) {
  using L = Layout<D>;
  constexpr int NST = L::NST;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {  // the tiles' swizzle needs it; there is no room to align by hand
    set_status(p.status, VSA_ERR_UNSUPPORTED);
    return;
  }
  // the joining kernel may be set up while this one runs
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  float* ml = reinterpret_cast<float*>(smem + L::kMLOff);
  PieceRing* items = reinterpret_cast<PieceRing*>(smem + L::kItemOff);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);

  const int tid = threadIdx.x;
  const int warp = tid / 32, lane = tid % 32;

  // the line needs the lengths from memory: first of all
  Walk walk(p, lane, warp == 3);

  if (warp == 0) {
    for (int i = lane; i < L::kNumBars; i += 32) {
      const uint32_t count = (i < L::kQFree || (i >= L::kPFull && i < L::kPFull + 2) ||
                              (i >= L::kLFull && i < L::kItFull))     ? 4u
                             : (i >= L::kOEmpty && i < L::kLFull)      ? 8u
                             : i >= L::kItEmpty                        ? 15u  // all warps but one
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
    tma_prefetch_desc(&tm_kp);
    tma_prefetch_desc(&tm_vp);
    tma_prefetch_desc(&tm_ks);
    tma_prefetch_desc(&tm_vs);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  auto next = [&](uint32_t& w, Piece& x) {
    return dense::get_item(items, bars + L::kItFull, bars + L::kItEmpty, w, x, lane, abort_flag, p.status);
  };

  if (warp < 4) {
    if (warp == 0) {
      // ===================== K and V tiles =====================
      const uint64_t pol_p = l2_policy_evict_last(), pol_s = l2_policy_evict_first();
      Piece x;
      uint32_t g = 0, n_got = 0;
      bool ok = true;
      while (ok && next(n_got, x)) {
        // the first instructions of the other warps, and Q, come before the stream
        // (64 requests of 512 keys: 47 us, 43)
        if (n_got == 1) ok = warp_wait(bars + L::kQFull, 0, abort_flag, p.status);
        if (lane == 0) {
          const bool own = x.b >= 0;
          const int b = own ? x.b : 0;
          for (int j = 0; ok && j < 2 * x.n; ++j, ++g) {
            const int st = (int)(g % NST);
            const uint32_t u = g / NST;
            if (u >= 1) ok = mbar_wait(bars + L::kEmpty + st, (u - 1) & 1, abort_flag, p.status);
            if (!ok) break;
            const bool order = split_rows(x) || j == 0 || j == 2 * x.n - 1;  // see place_k
            const bool is_v = order ? j & 1 : !(j & 1);
            const int key = 128 * (x.tile0 + (order ? j >> 1 : is_v ? (j >> 1) - 1 : (j + 1) >> 1));
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
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      }
      __syncwarp();
    } else if (warp == 2) {
      // ============ zero V rows past a segment's keys (what a cache holds there) ============
      Piece x;
      uint32_t g = 0, pre = 0, n_got = 0;
      while (next(n_got, x)) {
        g += 2 * x.n;
        const int len = x.kv_len - 128 * (x.tile0 + x.n - 1);
        if (len >= 128) continue;
        const int st = (int)((g - 1) % NST);
        if (!warp_wait(bars + L::kPre + st, (pre >> st) & 1, abort_flag, p.status)) break;
        pre ^= 1u << st;
        dense::zero_rows<128>(smem + L::kRingOff + st * L::kTile, L::DH, len, (len + 15) & ~15, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + L::kFull + st);
      }
    } else if (warp == 3) {
      // ===================== the line =====================
      if (blockIdx.x == 0)
        for (int b = lane; b < p.B; b += 32)
          if (p.lens[b] < 0 || p.lens[b] > p.suffix_cap) set_status(p.status, VSA_ERR_INDEX_RANGE);
      Piece x;
      uint32_t n = 0;
      bool ok = true;
      while (ok && walk.next(x))
        ok = dense::put_item(items, bars + L::kItFull, bars + L::kItEmpty, n++, x, lane, abort_flag, p.status);
      x.n = -1;
      if (ok) dense::put_item(items, bars + L::kItFull, bars + L::kItEmpty, n, x, lane, abort_flag, p.status);
    } else {
      // ===================== MMA issue: one thread =====================
      if (elect_one()) {
        // per slot: pieces whose products are issued, key tiles whose P has been
        // consumed.  (Scalars: an array indexed by the slot would live in memory.)
        uint32_t done0 = 0, done1 = 0, gs0 = 0, gs1 = 0;
        uint32_t g = 0, n_got = 0, n_q = 0;
        int n_s = 0;  // S products of the latest piece so far
        bool ok = true;
        auto wait = [&](int bar, uint32_t ph) {
          if (!mbar_wait(bars + bar, ph & 1, abort_flag, p.status)) ok = false;
        };
        // S(j) of slot s of the piece numbered n, whose ring tiles start at gx.  (All S of
        // a piece are issued before the first of the next one.)
        auto do_s = [&](const Piece& x, uint32_t n, int s, int j, uint32_t gx) {
          const int tile = slot_tile(x, s, j);
          const bool split = split_rows(x);
          const uint32_t gk = gx + place_k(x, tile);
          if (n_q == n) {  // the piece's first product
            wait(L::kQFull + (int)(n & 1), n >> 1);
            ++n_q;
            n_s = 0;
          }
          wait(L::kFull + (int)(gk % NST), gk / NST);
          if (!ok) return;
          tc_fence_after_sync();
          s_product<D>(tmem_base + 128u * s, sbase + L::kQOff + (split ? s : (int)(n & 1)) * L::kTile,
                     sbase + L::kRingOff + (gk % NST) * L::kTile);
          umma_commit(bars + L::kSFull + s);
          if (s == 1 || !split) umma_commit(bars + L::kEmpty + (int)(gk % NST));
          // The piece's last S: counted, for the slots' first S may be issued in either
          // order (slot 0 goes on first after a piece of more than 128 rows, and a slot that
          // found the piece not ready comes after the other), so that of two key tiles the
          // second may come first.  With its Q free too early the next 256 rows came over it.
          if (++n_s == (split ? 2 * x.n : x.n)) umma_commit(bars + L::kQFree + (int)(n & 1));
        };
        Piece x, y;
        auto next_one = [&](Piece& z) {
          return dense::get_item_one(items, bars + L::kItFull, bars + L::kItEmpty, n_got, z, abort_flag, p.status);
        };
        bool have = next_one(x);
        uint32_t n = 0;
        // the first S of slots 0, 1
        auto begin = [&](const Piece& z, uint32_t nz, int s, uint32_t gz) {
          if (ok && slot_tiles(z, s) > 0) do_s(z, nz, s, 0, gz);
        };
        // in the order of their tiles
        if (have) begin(x, 0, x.turn, 0);
        if (have) begin(x, 0, x.turn ^ 1, 0);
        while (ok && have) {
          const bool more = next_one(y);
          const uint32_t g_next = g + 2 * x.n;
          // a slot that is through with its tiles (or has none) goes on with the next
          // piece; where both slots read the same tiles, together and slot 0 first
          // (slot 1 releases the tile)
          const bool early = more && !split_rows(y);
          // ... if its Q and first tile are there: the products at hand do not wait for them
          auto ready = [&] {
            return (n_q > n + 1 || dense::slim::mbar_test_wait(bars + L::kQFull + (int)((n + 1) & 1), ((n + 1) >> 1) & 1)) &&
                   dense::slim::mbar_test_wait(bars + L::kFull + (int)(g_next % NST), (g_next / NST) & 1);
          };
          uint32_t later = 0;  // slots that go on with it after this piece's last product
          auto go_on = [&](int s, bool last) {
            if (last || ready()) begin(y, n + 1, s, g_next);
            else later |= 1u << s;
          };
          if (early && !split_rows(x) && x.n == 1) go_on(x.turn ^ 1, false);
          for (int i = 0; ok && i < x.n * (split_rows(x) ? 2 : 1); ++i) {
            // the slots in turn
            const int s = (i & 1) ^ x.turn, j = i >> 1, ns = slot_tiles(x, s);
            const int tile = slot_tile(x, s, j);
            const uint32_t gv = g + place_v(x, tile);
            const int st = (int)(gv % NST);
            wait(L::kFull + st, gv / NST);
            // the epilogue has emptied this slot's O
            const uint32_t done = s ? done1 : done0;
            if (j == 0 && done >= 1) wait(L::kOEmpty + s, done - 1);
            wait(L::kPFull + s, s ? gs1 : gs0);
            gs0 += s ^ 1;
            gs1 += s;
            if (!ok) break;
            tc_fence_after_sync();
            const int keys = x.kv_len - 128 * (x.tile0 + tile);
            pv_product<D>(tmem_base + kTmemO + D * s, tmem_base + 128u * s,
                        sbase + L::kRingOff + st * L::kTile, keys >= 128 ? 8 : (keys + 15) >> 4, j > 0);
            if (s == 1 || !split_rows(x)) umma_commit(bars + L::kEmpty + st);
            if (j + 1 < ns) {
              do_s(x, n, s, j + 1, g);
            } else {
              umma_commit(bars + L::kOFull + s);
              done0 += s ^ 1;
              done1 += s;
              if (early) go_on(s, i + 1 == x.n * (split_rows(x) ? 2 : 1) && !later);
            }
          }
          if (later) {  // in the order of their tiles
            if (later >> y.turn & 1) begin(y, n + 1, y.turn, g_next);
            if (later >> (y.turn ^ 1) & 1) begin(y, n + 1, y.turn ^ 1, g_next);
          }
          if (more && !early) begin(y, n + 1, 0, g_next);
          if (more && !early) begin(y, n + 1, 1, g_next);
          g = g_next;
          x = y;
          have = more;
          ++n;
        }
      }
      __syncwarp();
    }
  } else if (warp < 12) {
    // ============ softmax: one thread per row, or four (row_shift) ============
    const int s = (warp - 4) >> 2;
    const int wq = warp & 3;
    const uint32_t t_s = tmem_base + (uint32_t(wq * 32) << 16) + 128u * s;
    const uint32_t t_o = tmem_base + (uint32_t(wq * 32) << 16) + kTmemO + D * s;
    const float c = p.scale_log2;
    const uint64_t cc = pk2(c, c);
    uint32_t g = 0, n = 0, n_got = 0;
    bool ok = true;
    Piece x;
    while (ok && next(n_got, x)) {
      const int nt = slot_tiles(x, s);
      if (nt == 0) continue;  // a piece of one key tile leaves one slot nothing
      const int shift = row_shift(x);
      const bool any = (wq << shift) < slot_rows(x, s);  // this warp has rows
      // this thread's row, or the first of them
      const int row = (wq << shift) + (shift < 5 ? lane >> 2 : lane);
      auto keys_seen = [&](int r) {
        return x.kv_len + (x.b < 0 ? 0 : 1 - p.T + (256 * x.blk + (split_rows(x) ? 128 * s : 0) + r) % p.T);
      };
      const int limit = keys_seen(row);
      float m = -INFINITY;
      uint64_t l2 = pk2(0.f, 0.f);
      for (int j = 0; j < nt; ++j, ++g) {
        if (!warp_wait(bars + L::kSFull + s, g & 1, abort_flag, p.status)) { ok = false; break; }
        tc_fence_after_sync();
        const int key0 = 128 * (x.tile0 + slot_tile(x, s, j));
        if (any && shift == 3) {
          const int rem[1] = {min(128, limit - key0)};
          float mm[1] = {m};
          uint64_t ll[1] = {l2};
          dense::softmax_tile<D, 0, 1>(t_s, t_o, c, rem, __reduce_min_sync(0xffffffffu, rem[0]),
                                       __reduce_max_sync(0xffffffffu, rem[0]), j == 0, lane, mm, ll);
          m = mm[0], l2 = ll[0];
        } else if (any) {
          // columns before `whole` are seen by all of the warp's rows, from `none` on by none
          const int rem = min(128, limit - key0);
          const int whole = __reduce_min_sync(0xffffffffu, rem), none = __reduce_max_sync(0xffffffffu, rem);
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int q0 = 0; q0 < none; q0 += 32) {
            uint32_t v[32];
            tmem_ld32(t_s + q0, v);
            if (q0 + 32 > whole) {
#pragma unroll
              for (int q = 0; q < 32; ++q)
                if (q >= rem - q0) v[q] = __float_as_uint(-INFINITY);
            }
#pragma unroll
            for (int q = 0; q < 32; q += 8) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                mx[e] = fmax3(mx[e], __uint_as_float(v[q + 2 * e]), __uint_as_float(v[q + 2 * e + 1]));
            }
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
#pragma unroll 1
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
          // P's 16 columns of 32 bits lie over columns of S that were read before
#pragma unroll 1
          for (int q0 = 0; q0 < 128; q0 += 32) {
            uint32_t v[32], pk[16];
            if (q0 >= none) {
#pragma unroll
              for (int q = 0; q < 16; ++q) pk[q] = 0u;
              VSA_TMEM_ST16(t_s + q0 / 2, pk, 0);
              continue;
            }
            tmem_ld32(t_s + q0, v);
            if (q0 + 32 > whole) {
#pragma unroll
              for (int q = 0; q < 32; ++q)
                if (q >= rem - q0) v[q] = __float_as_uint(-INFINITY);
            }
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              float a, b;
              upk2(ffma2(pk2(__uint_as_float(v[2 * q]), __uint_as_float(v[2 * q + 1])), cc, nm2), a, b);
              a = fast_exp2(a);
              b = fast_exp2(b);
              l2 = fadd2(l2, pk2(a, b));
              pk[q] = pack_bf16x2(a, b);
            }
            VSA_TMEM_ST16(t_s + q0 / 2, pk, 0);
          }
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + L::kPFull + s);
      }
      if (!ok) break;
      // the epilogue has read the slot's previous maxima and sums
      if (n >= 1 && !warp_wait(bars + L::kOEmpty + s, (n - 1) & 1, abort_flag, p.status)) { ok = false; break; }
      ++n;
      float la, lb, l;
      if (shift < 5) {
        l = dense::quad_sum(l2);
      } else {
        upk2(l2, la, lb);
        l = la + lb;
      }
      // (four lanes may write the same)
      ml[s * 256 + row] = m;
      ml[s * 256 + 128 + row] = l;
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + L::kLFull + s);
      if (split_rows(x)) {
        // 256 rows to write: each slot's own warps, side by side
        if (!warp_wait(bars + L::kOFull + s, (n - 1) & 1, abort_flag, p.status)) { ok = false; break; }
        tc_fence_after_sync();
        const int rows = slot_rows(x, s);
        if (any) {
          const long long at = x.part * (x.b < 0 ? p.pfx_rows : p.sfx_rows) + 128 * s;
          if (row < rows) (x.b < 0 ? p.part_lse_p : p.part_lse_s)[at + row] = l == 0.f ? -INFINITY : m + __log2f(l);
          write_part<D>((x.b < 0 ? p.part_p : p.part_s) + at * D, 32 * wq, rows, lane, t_o, false,
                        l == 0.f ? 0.f : 1.f / l, 0.f);
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + L::kOEmpty + s);
      }
    }
  } else {
    // ===================== Q rows in, partial rows out (fp32) =====================
    const int wq = warp - 12;
    const uint32_t t_lane = tmem_base + (uint32_t(wq * 32) << 16) + kTmemO;
    uint32_t cs0 = 0, cs1 = 0;  // pieces of the slots
    uint32_t n_got = 0, freed = 0;  // pieces whose Q tiles are known to be free
    bool ok = true;
    // Rows of piece x (number n) into its Q tile or tiles: 16-byte chunks,
    // consecutive lanes along a row, into the 128-byte swizzle.  Rows past the
    // block keep what the tile held; only their own (unused) results depend on it.
    auto gather = [&](const Piece& x, uint32_t n, bool after_split) {
      const bool split = split_rows(x);
      // the tile's last reader: the piece before the previous one, or, where either
      // of this and the previous piece has both tiles, the previous one
      const uint32_t need = n == 0 ? 0u : (split || after_split) ? n : n - 1;
      for (; freed < need; ++freed)
        if (!warp_wait(bars + L::kQFree + (int)(freed & 1), (freed >> 1) & 1, abort_flag, p.status)) return false;
      constexpr int CH = D / 8, RPI = 32 / CH;  // chunks of a row, rows per access of the warp
      converge(warp);
      const int shift = row_shift(x);
      for (int r0 = wq << shift; r0 < x.rows; r0 += 128) {
        // this lane's row
        int i = 256 * x.blk + r0 + lane, b = x.b;
        if (b < 0) {
          b = i / p.rows_per_req;
          i -= b * p.rows_per_req;
        }
        const int gi = i / p.T;
        const long long off = b * p.q_st.b + (long long)(x.h * p.group + gi) * p.q_st.h + (long long)(i - gi * p.T) * p.q_st.s;
        uint8_t* qt = smem + L::kQOff + (split ? r0 >> 7 : (int)(n & 1)) * L::kTile;
        const int rows = min(1 << shift, x.rows - r0), ch = lane % CH;
#pragma unroll 4
        for (int r = 0; r < rows; r += RPI) {
          const int mine = r + lane / CH;
          const long long from = __shfl_sync(0xffffffffu, off, mine & 31);
          const int at = 32 * wq + mine;
          // all rows in flight at once, none of them in registers
          if (mine < rows)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                             smem_u32(qt + (ch >> 3) * 16384 + at * 128 + (((ch & 7) ^ (at & 7)) << 4))),
                         "l"(p.q + from + ch * 8)
                         : "memory");
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + L::kQFull + (int)(n & 1));
      return true;
    };
    Piece x, y;
    uint32_t n = 0;
    x.n = -1;  // no piece yet
    while (ok) {
      // the next piece's Q before this one's results
      const bool more = next(n_got, y);
      if (more && !gather(y, n, x.n > 0 && split_rows(x))) break;
      ++n;
      if (x.n < 0) {
        x = y;
        if (!more) break;
        continue;
      }
      const bool split = split_rows(x);
      const bool has0 = slot_tiles(x, 0) > 0, has1 = slot_tiles(x, 1) > 0;
      const bool two = has0 && has1;
#pragma unroll 1
      for (int s = 0; ok && s < 2; ++s) {
        if (s ? has1 : has0) {
          const uint32_t ph = (s ? cs1 : cs0) & 1;
          ok = warp_wait(bars + L::kLFull + s, ph, abort_flag, p.status) &&
               warp_wait(bars + L::kOFull + s, ph, abort_flag, p.status);
          if (!ok) break;
          cs0 += s ^ 1;
          cs1 += s;
        }
        // both slots are written together; a split piece's by its softmax warps,
        // but its maxima may be replaced only once these warps have passed here
        if (split) {
          if (lane == 0) mbar_arrive(bars + L::kOEmpty + s);
          continue;
        }
        if (s == 0) continue;
        tc_fence_after_sync();
        const int shift = row_shift(x), r0 = wq << shift, r_end = min(x.rows, r0 + (1 << shift));
        if (r0 < x.rows) {
          // weights of the slots' sums for this lane's row
          float w0 = 1.f, w1 = 0.f;
          const int row = r0 + lane;
          const int s0 = has0 ? 0 : 1;
          const float m0 = ml[s0 * 256 + row], l0 = ml[s0 * 256 + 128 + row];
          float top = m0, sum = l0;
          if (two) {
            const float m1 = ml[256 + row], l1 = ml[384 + row];
            top = fmaxf(m0, m1);
            const float ref = top == -INFINITY ? 0.f : top;
            w0 = fast_exp2(m0 - ref);
            w1 = fast_exp2(m1 - ref);
            sum = l0 * w0 + l1 * w1;
          }
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          const long long at = x.part * (x.b < 0 ? p.pfx_rows : p.sfx_rows);
          if (row < r_end) (x.b < 0 ? p.part_lse_p : p.part_lse_s)[at + row] = sum == 0.f ? -INFINITY : top + __log2f(sum);
          write_part<D>((x.b < 0 ? p.part_p : p.part_s) + at * D, r0, r_end, lane, t_lane + D * s0, two, w0 * inv, w1 * inv);
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          // for itself and in place of the softmax warps
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (has0) mbar_arrive(bars + L::kOEmpty);
            if (has1) mbar_arrive(bars + L::kOEmpty + 1);
          }
        }
      }
      x = y;
      if (!more) break;
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

// Suffix key tiles of the requests before each one, for batches whose lengths
// are too many for every warp of the other two kernels to add up: without it a
// call's time grew with the square of the batch.  One block, a thread per
// request, 1024 of them at a time.
constexpr int kTableThreads = 1024;
__global__ void __launch_bounds__(kTableThreads) prefix_table_kernel(const __grid_constant__ PrefixParams p) {
  __shared__ int warp_sum[kTableThreads / 32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int before = 0;  // of the requests before these 1024
  for (int b0 = 0; b0 < p.B; b0 += kTableThreads) {
    const int b = b0 + (int)threadIdx.x;
    const int mine = b < p.B ? key_tiles(suffix_len(p, b)) : 0;
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    int all = warp_sum[lane];  // as many warps as lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, all, o);
      if (lane >= o) all += v;
    }
    const int ahead = __shfl_sync(0xffffffffu, all, (warp + 31) & 31);  // warps before this one
    if (b < p.B) p.tiles_before[b] = before + (warp ? ahead : 0) + sum - mine;
    before += __shfl_sync(0xffffffffu, all, 31);
    __syncthreads();  // warp_sum is read
  }
  if (threadIdx.x == 0) p.tiles_before[p.B] = before;
}

// Joins the rows' partials: weights 2^(lse_i - max), fp32, in the order of the
// line.  A block has kJoinRows rows of one request and key head, one per warp.
constexpr int kJoinWarps = 4, kJoinRows = 4;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps)
    prefix_join_kernel(const __grid_constant__ PrefixParams p, int grid) {
  constexpr int E = D / 32;  // elements per lane
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int h = blockIdx.x % p.Hkv, b = blockIdx.x / p.Hkv;
  const Line line = make_line(p, lane, grid);
  const int tp = key_tiles(p.prefix_len), tb = key_tiles(suffix_len(p, b));
  const int before = suffix_tiles_before(p, b, lane);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the partial results are there
  const int row_end = min(p.rows_per_req, (int)(blockIdx.y + 1) * kJoinRows);
  for (int row = blockIdx.y * kJoinRows + warp; row < row_end; row += kJoinWarps) {
    float m = -INFINITY, l = 0.f, o[E] = {};
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {
      // the segment's tiles, its first partial and the row in it
      const int tiles = kind ? tb : tp;
      if (tiles == 0) continue;
      const int r = kind ? row : b * p.rows_per_req + row;
      const int blk = r >> 8;
      const int t0 = h * line.per_head + (kind ? line.pfx * tp + line.sfx * before : 0) + blk * line.heavy * tiles;
      const int w = tile_units(line, kind ? p.rows_per_req : p.B * p.rows_per_req, blk);
      const int c0 = cta_of(line, t0), count = cta_of(line, t0 + w * (tiles - 1)) - c0 + 1;
      const long long seg = kind ? ((long long)h * p.B + b) * p.sfx_blocks + blk : (long long)h * p.pfx_blocks + blk;
      const int rows = kind ? p.sfx_rows : p.pfx_rows;
      const long long first = (seg + c0) * rows + (r & 255);
      const float* lse = kind ? p.part_lse_s : p.part_lse_p;
      const float* part = (kind ? p.part_s : p.part_p) + lane * E;
      for (int i0 = 0; i0 < count; i0 += 32) {
        const float mine = i0 + lane < count ? lse[first + (long long)(i0 + lane) * rows] : -INFINITY;
        // nothing seen in any of them (a NaN is not that, though the maximum passes over it)
        if (__all_sync(0xffffffffu, mine == -INFINITY)) continue;
        float top = mine;
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
        const float nm = fmaxf(m, top), a = fast_exp2(m - nm);
        m = nm;
        l *= a;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= a;
        const int here = min(32, count - i0);
#pragma unroll 4
        for (int i = 0; i < here; ++i) {
          const float x = __shfl_sync(0xffffffffu, mine, i);
          const float w = fast_exp2(x - nm);
          const float* src = part + (first + (long long)(i0 + i) * rows) * D;
          float v[E];
          if (E == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(src);
          else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(src);
          // a part of which the row saw nothing weighs nothing, whatever its v left there (0 * NaN)
          const bool none = x == -INFINITY;
          l += none ? 0.f : w;
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] = none ? o[e] : fmaf(w, v[e], o[e]);
        }
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int g = row / p.T, t = row - g * p.T;
    const int head = h * p.group + g;
    __nv_bfloat16* out = p.out + b * p.out_st.b + head * p.out_st.h + (long long)t * p.out_st.s + lane * E;
    uint32_t pk[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) pk[e] = pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
    if (E == 4) *reinterpret_cast<uint2*>(out) = make_uint2(pk[0], pk[1]);
    else *reinterpret_cast<uint32_t*>(out) = pk[0];
    if (p.lse && lane == 0)
      p.lse[((long long)b * p.Hq + head) * p.T + t] =
          l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
  }
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
  p->pfx_rows = all < 256 ? all : 256;
  p->sfx_rows = p->rows_per_req < 256 ? p->rows_per_req : 256;
}

// Partial results of each kind: segments + CTAs, of a block's rows each.
static size_t parts_of(long long segments, int rows) {
  return (size_t)(segments + kPrefixGrid) * rows;
}
static size_t a256(size_t x) { return (x + 255) & ~size_t(255); }

// Requests from which on their key tiles are added up once, by a kernel of its
// own (64 query heads over 8, 1000 shared and up to 200 own keys, us by the warps
// and by the kernel: 64 requests 37, 41; 200: 94, 97; 256: 121, 121; 512: 211, 205;
// 4096: 2055, 1548; 65536 with 8 heads over 1: 19550, 2118).
#ifndef PREFIX_TABLE_REQUESTS
#define PREFIX_TABLE_REQUESTS 512
#endif

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
  p->tiles_before = nullptr;
  if (sfx && p->B >= PREFIX_TABLE_REQUESTS) p->tiles_before = reinterpret_cast<int*>(take((size_t)p->B + 1));
  return off;
}

template <int D>
static int launch_prefix_t(PrefixParams p, const CUtensorMap* m, cudaStream_t stream) {
  using L = prefix::Layout<D>;
  auto kern = prefix::prefix_attn_kernel<D>;
  static KernelReady ready;
  const int rc = ready.check(reinterpret_cast<const void*>(kern), (int)L::kAlloc);
  if (rc != VSA_OK) return rc;
  // at most one CTA per key tile there can be
  const long long cap = (long long)p.Hkv * ((long long)p.pfx_blocks * ((p.prefix_len + 127LL) / 128) +
                                            (long long)p.B * p.sfx_blocks * ((p.suffix_cap + 127LL) / 128));
  const int grid = cap < kPrefixGrid ? (int)(cap > 0 ? cap : 1) : kPrefixGrid;
  // 20 us per tile of a CTA's share, ten times what one takes: a wait may last a piece
  p.item_us = (int)std::min(20 * (cap / grid + 1), 1000000000LL);
  if (p.tiles_before) prefix::prefix_table_kernel<<<1, prefix::kTableThreads, 0, stream>>>(p);
  kern<<<grid, prefix::kThreads, L::kAlloc, stream>>>(m[0], m[1], m[2], m[3], p);
  if (cudaGetLastError() != cudaSuccess) return VSA_ERR_CUDA;
  // set up while the attention kernel runs; waits for it before it reads partial results
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.B * p.Hkv), (unsigned)((p.rows_per_req + prefix::kJoinRows - 1) / prefix::kJoinRows));
  cfg.blockDim = dim3(32 * prefix::kJoinWarps);
  cfg.stream = stream;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefix::prefix_join_kernel<D>, p, grid) == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
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

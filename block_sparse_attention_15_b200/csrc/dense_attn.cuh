// What the dense-attention kernels (forward, dq, dk/dv) share: the packed
// sequences of a launch, the order in which their tiles are worked on, and the
// tile loads.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include <type_traits>

#include "dense_launch.h"
#include "vsa_device.cuh"

namespace vsa {
namespace dense {

// The waits of vsa_device.cuh with their polling out of line: a kernel waits in
// dozens of places, and with the polling inlined its code (90-115 KB) did not
// stay in the instruction caches.
namespace slim {
// A wait may last as long as the longest work item: abort_flag[1] holds the
// microseconds that adds to the limit.
static __device__ __noinline__ bool mbar_poll(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                              int* status) {
  unsigned long long t0 = 0;
  for (;;) {
    // (a failed try has slept for some microseconds, or until the phase completed)
    for (int i = 0; i < 16; ++i)
      if (mbar_try_wait_sleep(bar, parity, kPollSleepNs)) return true;
    if (abort_flag[0]) return false;
    if (status && *reinterpret_cast<volatile int*>(status) == VSA_ERR_DEVICE_TIMEOUT) {
      abort_flag[0] = 1;
      return false;
    }
    const unsigned long long now = global_timer_ns();
    if (t0 == 0) t0 = now;
    else if (now - t0 > kWaitTimeoutNs + 1000ull * (unsigned)abort_flag[1]) {
      set_status(status, VSA_ERR_DEVICE_TIMEOUT);
      abort_flag[0] = 1;
      return false;
    }
  }
}
static __device__ __noinline__ bool warp_poll(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                              int* status) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = mbar_poll(bar, parity, abort_flag, status) ? 1 : 0;
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}
// Whether the phase is complete, at once.
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  return mbar_try_wait(bar, parity) || mbar_poll(bar, parity, abort_flag, status);
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || warp_poll(bar, parity, abort_flag, status);
}
}  // namespace slim

// Unit i of a launch, the long ones first.  The table's first sequences are flat
// (their units cost about the same): by descending cost, one after the other.
// The others have units whose cost grows with their rank t (tile t of a causal
// sequence has about t + 1 tiles to read): sorted by their unit counts
// n_0 >= n_1 >= ..., their units are taken by descending rank, every sequence
// that has a unit of that rank in turn.  The ranks n_r .. n_{r-1} - 1 are those
// that exactly r of them have.
struct Unit {
  int seq;   // index into DenseSeqs::seq
  int rank;  // 0 .. units[seq] - 1
};

__device__ __forceinline__ Unit find_unit(const DenseSeqs& t, int i) {
  const bool flat = i < t.first[t.n_flat];
  // the last entry of first[] that is not past i
  int lo = flat ? 0 : t.n_flat + 1, hi = flat ? t.n_flat - 1 : t.n;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  const int o = i - t.first[lo];
  Unit u;
  if (flat) {
    u.seq = lo;
    u.rank = t.units[lo] - 1 - o;
  } else {
    const int r = lo - t.n_flat;
    u.seq = t.n_flat + o % r;
    u.rank = t.units[lo - 1] - 1 - o / r;
  }
  return u;
}

// Blocks of the grid are work items.  Those that find an SM at launch stay on it
// and take over blocks that have not started (cluster launch control), in the
// grid's order, until none is left: an SM that is through early takes more,
// without a counter in memory.  One warp asks; `reply` is 16 bytes of shared
// memory, `bar` counts one arrival.
struct Takeover {
  uint64_t* bar;
  uint4* reply;
  uint32_t asked;

  __device__ __forceinline__ void ask(int lane) {
    if (lane == 0) {
      mbar_arrive_expect_tx(bar, 16);
      asm volatile(
          "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
              smem_u32(reply)),
          "r"(smem_u32(bar))
          : "memory");
    }
    __syncwarp();
  }
  // The block taken over, -1: none is left (and none may be asked for again).
  __device__ __forceinline__ int answer(volatile int* abort_flag, int* status) {
    if (!slim::warp_wait(bar, asked++ & 1, abort_flag, status)) return -1;
    uint32_t got, block;
    asm volatile(
        "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
        "ld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}\n"
        : "=r"(got), "=r"(block)
        : "r"(smem_u32(reply))
        : "memory");
    // the reply is read before the next one may be written
    fence_proxy_async_smem();
    __syncwarp();
    return got ? (int)block : -1;
  }
};

// Work items of a CTA: one warp finds them (searches and divisions of a few
// hundred cycles) and hands them to the others through a ring in shared memory.
// (Two slots where items are taken over: no CTA holds many that others could do.)
template <typename Item, int N>
struct alignas(16) ItemRing {
  static constexpr int kSlots = N;
  Item item[N];
};

// The finder's side, whole warp: the w-th item, or the end mark (n < 0).
template <typename Item, int N>
__device__ __forceinline__ bool put_item(ItemRing<Item, N>* ring, uint64_t* full, uint64_t* empty, uint32_t w,
                                         const Item& x, int lane, volatile int* abort_flag, int* status) {
  const int slot = (int)(w % N);
  if (w >= (uint32_t)N && !slim::warp_wait(empty + slot, (w / N - 1) & 1, abort_flag, status))
    return false;
  if (lane == 0) {
    ring->item[slot] = x;
    mbar_arrive(full + slot);
  }
  __syncwarp();
  return true;
}

// The other warps' side: false at the end.
template <typename Item, int N>
__device__ __forceinline__ bool get_item(const ItemRing<Item, N>* ring, uint64_t* full, uint64_t* empty, uint32_t& w,
                                         Item& x, int lane, volatile int* abort_flag, int* status) {
  const int slot = (int)(w % N);
  if (!slim::warp_wait(full + slot, (w / N) & 1, abort_flag, status)) return false;
  x = ring->item[slot];
  __syncwarp();
  if (lane == 0) mbar_arrive(empty + slot);
  ++w;
  return x.n >= 0;
}

// The same for a role that one thread plays.
template <typename Item, int N>
__device__ __forceinline__ bool get_item_one(const ItemRing<Item, N>* ring, uint64_t* full, uint64_t* empty,
                                             uint32_t& w, Item& x, volatile int* abort_flag, int* status) {
  const int slot = (int)(w % N);
  if (!slim::mbar_wait(full + slot, (w / N) & 1, abort_flag, status)) return false;
  x = ring->item[slot];
  mbar_arrive(empty + slot);
  ++w;
  return x.n >= 0;
}

// 64 head dims x box rows of a [H, S, D] view through its tile map.
__device__ __forceinline__ void load_rows(void* dst, const CUtensorMap* map, TmaAxes ax,
                                          uint64_t* bar, int d0, int s, int h, int b,
                                          uint64_t hint) {
  const int c1 = ax.s == 1 ? s : (ax.h == 1 ? h : b);
  const int c2 = ax.s == 2 ? s : (ax.h == 2 ? h : b);
  const int c3 = ax.s == 3 ? s : (ax.h == 3 ? h : b);
  tma_load_4d(dst, map, bar, d0, c1, c2, c3, hint);
}

// Rows `from` .. `to` - 1 of a tile of `slabs` 64-column slabs (ROWS rows of
// 128 bytes each) become zero: the warp's lanes write 16 bytes each.  The
// swizzle only permutes a row's eight 16-byte chunks, so it can be ignored.
template <int ROWS>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int slabs, int from, int to, int lane) {
  const int n = (to - from) * 8;
  for (int sl = 0; sl < slabs; ++sl)
    for (int i = lane; i < n; i += 32)
      *reinterpret_cast<uint4*>(tile + sl * (ROWS * 128) + from * 128 + i * 16) =
          make_uint4(0u, 0u, 0u, 0u);
}

// 16 TMEM lanes x 32 fp32 columns: register 4 i + 2 b + e holds lane
// threadIdx / 4 + 8 b, column 8 i + 2 (threadIdx % 4) + e.
template <int N>
__device__ __forceinline__ void tmem_ld_16x256(uint32_t taddr, uint32_t (&r)[N], int o) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[o + 0]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]),
        "=r"(r[o + 6]), "=r"(r[o + 7]), "=r"(r[o + 8]), "=r"(r[o + 9]), "=r"(r[o + 10]), "=r"(r[o + 11]),
        "=r"(r[o + 12]), "=r"(r[o + 13]), "=r"(r[o + 14]), "=r"(r[o + 15])
      : "r"(taddr));
}

// 16 TMEM lanes x 64 fp32 columns, as above with twice the columns; and back.
__device__ __forceinline__ void tmem_ld_16x256_64(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st_16x256(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 16 TMEM lanes x 32 columns of 32 bits: register 2 i + b holds lane
// threadIdx / 4 + 8 b, column 4 i + threadIdx % 4.
__device__ __forceinline__ void tmem_st_16x128_32(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// 2^x for a pair of floats on the FMA pipe, as exp2_fma2 has it (the same cubic),
// for any x < 128: NaN gives NaN, and what is below -126.5, -infinity too, gives
// 0.  The clamp keeps NaN; 2^j is made a number of its own, whose exponent field is
// 0 at j = -127, and multiplied by, which keeps NaN as well.  (The sparse kernels'
// form adds j to the exponent field, one instruction less, and turns NaN and
// -infinity into 2^-120.)
__device__ __forceinline__ uint64_t exp2_fma2_any(float x0, float x1) {
  constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer
  float c0, c1;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(c0) : "f"(x0), "f"(-127.f));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(c1) : "f"(x1), "f"(-127.f));
  const uint64_t xx = pk2(c0, c1);
  const uint64_t t = fadd2(xx, pk2(kRound, kRound));
  const uint64_t j = fadd2(t, pk2(-kRound, -kRound));
  const uint64_t f = ffma2(j, pk2(-1.f, -1.f), xx);
  uint64_t q = ffma2(f, pk2(0x1.c3f760p-5f, 0x1.c3f760p-5f), pk2(0x1.f0de1ap-3f, 0x1.f0de1ap-3f));
  q = ffma2(q, f, pk2(0x1.62f31ap-1f, 0x1.62f31ap-1f));
  q = ffma2(q, f, pk2(0x1.fff692p-1f, 0x1.fff692p-1f));
  float t0, t1;
  upk2(t, t0, t1);  // their low bits hold j
  return fmul2(q, pk2(__int_as_float((__float_as_int(t0) << 23) + 0x3f800000),
                      __int_as_float((__float_as_int(t1) << 23) + 0x3f800000)));
}

// Largest excess (log2 units) of a logit over its row's reference max that is
// exponentiated without moving the reference: probabilities stay below 2^8.
constexpr float kRefresh = 8.f;

// One 128-key tile of the online softmax, by a warp that has 8 NB rows of the
// query tile (TMEM lanes from t_s's on): a thread has rows lane / 4 + 8 b, b < NB,
// and a quarter of their columns.  In the forward kernel two warps share the 32
// lanes that each may reach, so that a slot's softmax is eight warps' work.  A row
// stays within one warp: its max takes two shuffles, its sum none until the end.
// S is read twice (a load takes 50 cycles) rather than kept in 64 registers.
//   rem[b]: columns of the tile that row b sees; whole / none: the least and the
//   largest of those over the warp, at most 128
//   m, l2: the rows' reference max (log2 units) and partial sums; O is rescaled
//   when a reference moves (S complete implies the PV before it is: one thread
//   issued both, in order)
// POLY of eight column pairs take their exponential on the FMA pipe.
template <int D, int POLY, int UNROLL, int NB>
__device__ __forceinline__ void softmax_tile(uint32_t t_s, uint32_t t_o, float c, const int (&rem)[NB], int whole,
                                             int none, bool first, int lane, float (&m)[NB], uint64_t (&l2)[NB]) {
  const int col0 = 2 * (lane & 3);
  auto mask = [&](uint32_t (&v)[32], int q0) {
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (((k >> 1) & 1) < NB && 8 * (k >> 2) + (k & 1) >= rem[(k >> 1) & (NB - 1)] - q0 - col0) v[k] = 0xff800000u;  // -inf
  };
  float mx[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) mx[b] = -INFINITY;
#pragma unroll UNROLL
  for (int q0 = 0; q0 < 128; q0 += 64) {
    if (q0 >= none) break;
    uint32_t v[32];
    tmem_ld_16x256_64(t_s + q0, v);
    if (q0 + 64 > whole) mask(v, q0);
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
      mx[0] = fmax3(mx[0], __uint_as_float(v[k]), __uint_as_float(v[k + 1]));
      if (NB == 2) mx[NB - 1] = fmax3(mx[NB - 1], __uint_as_float(v[k + 2]), __uint_as_float(v[k + 3]));
    }
  }
  float nm[NB];
  bool move = false;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    mx[b] = fmaxf(mx[b], __shfl_xor_sync(0xffffffffu, mx[b], 1));
    mx[b] = fmaxf(mx[b], __shfl_xor_sync(0xffffffffu, mx[b], 2)) * c;
    const bool up = mx[b] > m[b] + kRefresh;
    nm[b] = up ? mx[b] : m[b];
    move = move || up;
  }
  if (__any_sync(0xffffffffu, move)) {
    float a[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      // 1 where the reference stays; 0 while nothing was seen (O and the sum are 0)
      a[b] = m[b] == -INFINITY ? 0.f : fast_exp2(m[b] - nm[b]);
      float la, lb;
      upk2(l2[b], la, lb);
      l2[b] = pk2(la * a[b], lb * a[b]);
      m[b] = nm[b];
    }
    if (!first) {
#pragma unroll 1
      for (int q0 = 0; q0 < D; q0 += 32) {
        uint32_t ov[16];
        tmem_ld_16x256(t_o + q0, ov, 0);
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (((k >> 1) & 1) < NB) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * a[(k >> 1) & (NB - 1)]);
        tmem_st_16x256(t_o + q0, ov);
      }
    }
  }
  // probabilities 2^(s c - m): bf16 pairs for the tensor core, fp32 sums.  P's 32
  // columns per step lie over columns of S that were read before.
  const uint64_t cc = pk2(c, c);
  uint64_t nm2[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const float ref = m[b] == -INFINITY ? 0.f : -m[b];  // nothing seen yet: all -inf, all 0
    nm2[b] = pk2(ref, ref);
  }
#pragma unroll UNROLL
  for (int q0 = 0; q0 < 128; q0 += 64) {
    uint32_t pk[16];
    if (q0 >= none) {
#pragma unroll
      for (int k = 0; k < 16; ++k) pk[k] = 0u;
      tmem_st_16x128_32(t_s + q0 / 2, pk);
      continue;
    }
    uint32_t v[32];
    tmem_ld_16x256_64(t_s + q0, v);
    auto probs = [&](auto mk) {
      constexpr bool kMask = decltype(mk)::value;
      if (kMask) mask(v, q0);
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        if ((k & 1) >= NB) {  // a row of none of this warp's
          pk[k] = 0u;
          continue;
        }
        const int w = k & (NB - 1);
        float a, b;
        upk2(ffma2(pk2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), cc, nm2[w]), a, b);
        if (!kMask && (k & 7) < POLY) {
          upk2(exp2_fma2_any(a, b), a, b);
        } else {
          a = fast_exp2(a);
          b = fast_exp2(b);
        }
        l2[w] = fadd2(l2[w], pk2(a, b));
        pk[k] = pack_bf16x2(a, b);
      }
    };
    if (q0 + 64 > whole) probs(std::true_type{});
    else probs(std::false_type{});
    tmem_st_16x128_32(t_s + q0 / 2, pk);
  }
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// The whole sum of a row whose partial sums four neighbouring lanes have.
__device__ __forceinline__ float quad_sum(uint64_t l2) {
  float la, lb;
  upk2(l2, la, lb);
  float l = la + lb;
  l += __shfl_xor_sync(0xffffffffu, l, 1);
  return l + __shfl_xor_sync(0xffffffffu, l, 2);
}

// S = Q . K^T: M = N = 128, K = D; tiles are [D / 64][128 rows][128 B].
template <int D>
__device__ __forceinline__ void issue_s(uint32_t tmem_d, uint32_t q_base, uint32_t k_base) {
  constexpr uint32_t idesc = make_idesc_bf16(128, 128, false, false);
  const uint64_t a0 = make_sdesc_sw128(q_base, 16u, 1024u);
  const uint64_t b0 = make_sdesc_sw128(k_base, 16u, 1024u);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint64_t off = (uint64_t)(((kk / 4) * 16384 + (kk % 4) * 32) >> 4);
    umma_bf16(tmem_d, a0 + off, b0 + off, idesc, kk > 0 ? 1u : 0u);
  }
}

// O (+)= P . V over the first 16 * steps keys of the tile.
template <int D>
__device__ __forceinline__ void issue_pv(uint32_t tmem_o, uint32_t tmem_p, uint32_t v_base,
                                         int steps, bool accumulate) {
  constexpr uint32_t idesc = make_idesc_bf16(128, D, false, true);
  const uint64_t b0 = make_sdesc_sw128(v_base, 16384u, 1024u);
  if (steps == 8) {
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
      umma_bf16_tmem_a(tmem_o, tmem_p + 8u * kk, b0 + (uint64_t)((kk * 2048) >> 4), idesc,
                       (accumulate || kk > 0) ? 1u : 0u);
  } else {
    for (int kk = 0; kk < steps; ++kk)
      umma_bf16_tmem_a(tmem_o, tmem_p + 8u * kk, b0 + (uint64_t)((kk * 2048) >> 4), idesc,
                       (accumulate || kk > 0) ? 1u : 0u);
  }
}

// A launch whose waits ran out leaves only after copies that may still be in
// flight have landed (they take microseconds).
__device__ __forceinline__ void settle_after_abort(volatile int* abort_flag) {
  if (abort_flag[0])
    for (int i = 0; i < 20; ++i) __nanosleep(100000);
}

}  // namespace dense
}  // namespace vsa

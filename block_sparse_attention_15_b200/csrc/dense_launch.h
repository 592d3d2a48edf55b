// Host-side parameter blocks and launchers of the dense-attention kernels.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "vsa_launch.h"

namespace vsa {

// Sequences one launch takes; longer batches are split over launches.  (With 128
// a launch's parameters stay below 4 KB: 3.2 us of host time instead of 4.0.)
constexpr int kDenseMaxSeqs = 128;

// Packed sequences of one launch, passed by value (so a captured launch keeps
// its lengths).  3.1 KB.
struct DenseSeqs {
  int n, n_flat;
  int n_units;                      // of all sequences (what a unit is, each kernel says)
  int4 seq[kDenseMaxSeqs];          // first q row, q rows, first kv row, kv rows
  int units[kDenseMaxSeqs];         // units of the sequence
  // [0, n_flat): units before the sequence; [n_flat]: units of the flat ones;
  // [n_flat + r]: units before the ranks that exactly r of the others have
  int first[kDenseMaxSeqs + 1];
};

struct DenseParams {
  __nv_bfloat16* out;
  Strides3 out_st;                  // b unused
  float* lse;                       // [Hq, lse_seq] or null
  long long lse_seq;
  TmaAxes q_ax, k_ax, v_ax;
  int Hq, Hkv, group;               // group = Hq / Hkv
  int causal;
  int slots;                        // row tiles per work item: 1 or 2
  int item_us;                      // see item_microseconds
  float scale_log2;
  int* status;
};

// One call's tensors: [H, S, D] views (Strides3::b unused).
struct DenseTensors {
  const void *q, *k, *v;
  Strides3 q_st, k_st, v_st;
  long long q_seq, kv_seq;          // rows of the q and k/v views
};

// Host cumulative lengths of a batch (checked by the caller).
struct DenseBatch {
  const int32_t* cu_q;
  const int32_t* cu_kv;
  int n;
  // sequences i0 .. of at most kDenseMaxSeqs, as DenseSeqs::seq entries
  int chunk(int i0, int4* seqs) const;
};

// Once per device: the kernel's shared memory limit is raised.
struct KernelReady {
  std::atomic<unsigned long long> done{0};
  int check(const void* kern, int smem);
};

int device_sm_count();
// 20 us per tile of the longest work item (10 times what one takes), which a wait
// on an item may last on top of the waits' own limit: over the keys of a sequence,
// or over its rows in each head of a group.
int item_microseconds(const DenseBatch& b, bool over_rows, int group);
// Fills the table (dropping sequences without units).  `flat_cost` of a sequence:
// the cost of each of its units where they cost about the same, else 0; all in
// the order of `seqs`, the units' sum below 2^30.
void fill_dense_seqs(DenseSeqs* t, const int4* seqs, const int* units, const int* flat_cost, int n);
int launch_dense_fwd(const DenseParams& p, const DenseTensors& t, const DenseBatch& b, int D,
                     cudaStream_t stream);

// Gradients (dense_bwd.cu): one launch for dq (and delta), one for dk and dv.
struct DenseBwdParams {
  __nv_bfloat16 *dq, *dk, *dv;
  Strides3 dq_st, dk_st, dv_st;
  const float* lse;                 // [Hq, lse_seq]
  float* delta;                     // [Hq, lse_seq] workspace
  float* part;                      // [parts][dk, dv][Hkv][part_rows][D] workspace, see dkv_parts
  int parts, part_row0, part_rows;  // rows part_row0 .. of k and v
  long long lse_seq;
  TmaAxes q_ax, k_ax, v_ax, do_ax, o_ax;
  int Hq, Hkv, group;
  int causal;
  int item_us;                      // see item_microseconds
  float scale, scale_log2;
  int* status;
};
// CTAs that share a key tile's walk over the query rows: more than one where the
// key tiles of a launch (n sequences) would leave SMs idle for long.
int dkv_parts(const int4* seqs, int n, int Hq, int Hkv, bool causal);
size_t dense_bwd_workspace(const DenseBatch& b, int Hq, int Hkv, int D, long long q_rows, bool causal);
int launch_dense_bwd(const DenseBwdParams& p, const DenseTensors& t, const void* out, Strides3 out_st,
                     const void* dout, Strides3 do_st, const DenseBatch& b, int D, cudaStream_t stream);

// Shared-prefix decoding (prefix_attn.cu).  CTAs of its attention kernel: one
// per SM, and a constant, so that the workspace and the split of the work (and
// with it the rounding) depend on the arguments alone.
constexpr int kPrefixGrid = 148;
struct PrefixParams {
  const __nv_bfloat16* q;           // [B, Hq, T, D] view
  __nv_bfloat16* out;
  Strides3 q_st, out_st;
  float* lse;                       // [B, Hq, T] or null
  const int32_t* lens;              // [B] device
  int B, Hq, Hkv, T, prefix_len, suffix_cap;
  float scale_log2;
  int* status;
  int item_us;                      // microseconds that the longest share may take
  // filled by prefix_shape
  int group, rows_per_req;          // Hq / Hkv, group * T
  int pfx_blocks, sfx_blocks;       // row blocks of 256 of a prefix / suffix segment
  int pfx_rows, sfx_rows;           // rows of a partial result
  // workspace
  float *part_p, *part_s, *part_lse_p, *part_lse_s;
  int* tiles_before;                // [B + 1] suffix key tiles of the requests before one, or null
  TmaAxes kp_ax, vp_ax, ks_ax, vs_ax;
};
struct PrefixTensors {
  const void *k_prefix, *v_prefix, *k_suffix, *v_suffix;
  Strides3 kp_st, vp_st, ks_st, vs_st;
};
void prefix_shape(PrefixParams* p);
// Lays the workspace out at `base` (may be null to size it); its bytes.
size_t prefix_workspace(PrefixParams* p, int D, void* base);
int launch_prefix(const PrefixParams& p, const PrefixTensors& t, int D, cudaStream_t stream);

}  // namespace vsa

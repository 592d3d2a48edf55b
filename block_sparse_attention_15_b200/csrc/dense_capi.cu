// C ABI of the dense-attention entries (vsa.h): argument checks and launches.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "dense_launch.h"
#include "vsa.h"
#include "vsa_launch.h"

namespace vsa {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A [H, S, D] view: strides of axes longer than one are positive multiples of
// 8 elements (16 bytes: tile maps and 16-byte accesses).
bool view_ok(const vsa_strides& s, long long H, long long S) {
  auto ok = [](long long stride, long long extent) {
    return extent <= 1 || (stride > 0 && stride % 8 == 0);
  };
  return ok(s.head, H) && ok(s.seq, S);
}

Strides3 to3(const vsa_strides& s) { return Strides3{s.batch, s.head, s.seq}; }

// Cumulative lengths: start at 0, never fall, end within the tensor's rows.
bool cumulative_ok(const int32_t* cu, int n, long long rows) {
  if (cu[0] != 0) return false;
  for (int i = 0; i < n; ++i)
    if (cu[i + 1] < cu[i]) return false;
  return cu[n] <= rows;
}

constexpr long long kMaxRows = 0x7FFFFFFFLL - 256;  // tile coordinates are 32-bit

int check_dense(int n_seqs, const int32_t* cu_q, const int32_t* cu_kv, int Hq, int Hkv, int D,
                int64_t q_rows, int64_t kv_rows, float scale) {
  if (!cu_q || !cu_kv || Hq <= 0 || Hkv <= 0 || q_rows < 0 || kv_rows < 0 || !(scale == scale))
    return VSA_ERR_INVALID_ARG;
  if (n_seqs <= 0) return VSA_ERR_SHAPE;
  if (D != 64 && D != 128) return VSA_ERR_UNSUPPORTED;
  if (Hq % Hkv) return VSA_ERR_SHAPE;
  if (q_rows > kMaxRows || kv_rows > kMaxRows || Hq > 65535) return VSA_ERR_UNSUPPORTED;
  if (!cumulative_ok(cu_q, n_seqs, q_rows) || !cumulative_ok(cu_kv, n_seqs, kv_rows)) return VSA_ERR_SHAPE;
  return VSA_OK;
}

bool view4_ok(const vsa_strides& s, long long B, long long H, long long S) {
  return view_ok(s, H, S) && (B <= 1 || (s.batch > 0 && s.batch % 8 == 0));
}

// Sizes of a shared-prefix call; fills the shape fields of `p`.
int check_prefix(PrefixParams* p, int B, int Hq, int Hkv, int T, int D, int64_t prefix_len,
                 int64_t suffix_cap) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || T < 0 || prefix_len < 0 || suffix_cap < 0) return VSA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return VSA_ERR_UNSUPPORTED;
  if (Hq % Hkv) return VSA_ERR_SHAPE;
  // rows, and the key tiles of all key heads, are counted in 32 bits
  const long long per_req = (long long)(Hq / Hkv) * T;
  if (prefix_len > kMaxRows || suffix_cap > kMaxRows || Hq > 65535 || per_req > (1 << 24) ||
      B * per_req > (1 << 28) || (long long)B * Hq * T > (1 << 30))
    return VSA_ERR_UNSUPPORTED;
  const long long tiles = (B * per_req + 255) / 256 * ((prefix_len + 127) / 128) +
                          (long long)B * ((per_req + 255) / 256) * ((suffix_cap + 127) / 128);
  if (tiles > (1 << 29) / Hkv || (per_req + 3) / 4 > 65535) return VSA_ERR_UNSUPPORTED;
  p->B = B;
  p->Hq = Hq;
  p->Hkv = Hkv;
  p->T = T;
  p->prefix_len = (int)prefix_len;
  p->suffix_cap = (int)suffix_cap;
  prefix_shape(p);
  return VSA_OK;
}

void contiguous_layout(vsa_dense_layout* L, int64_t q_rows, int64_t kv_rows, int D) {
  const vsa_strides q{0, q_rows * D, D}, kv{0, kv_rows * D, D};
  L->q = L->out = L->dout = L->dq = q;
  L->k = L->v = L->dk = L->dv = kv;
}

}  // namespace
}  // namespace vsa

using namespace vsa;

extern "C" {

int dense_attn_varlen(const void* q, const void* k, const void* v, const vsa_dense_layout* layout,
                      const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_kv, int n_seqs, int Hq,
                      int Hkv, int D, int64_t q_rows, int64_t kv_rows, int causal, float scale,
                      void* out, float* lse, void* stream) {
  int rc = check_dense(n_seqs, cu_seqlens_q, cu_seqlens_kv, Hq, Hkv, D, q_rows, kv_rows, scale);
  if (rc != VSA_OK) return rc;
  if (cu_seqlens_q[n_seqs] == 0) return VSA_OK;  // no rows
  const bool keys = cu_seqlens_kv[n_seqs] > 0;
  if (!q || !out || (keys && (!k || !v))) return VSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || (keys && (!aligned16(k) || !aligned16(v))))
    return VSA_ERR_INVALID_ARG;
  vsa_dense_layout L;
  if (layout) L = *layout;
  else contiguous_layout(&L, q_rows, kv_rows, D);
  if (!view_ok(L.q, Hq, q_rows) || !view_ok(L.out, Hq, q_rows) ||
      (keys && (!view_ok(L.k, Hkv, kv_rows) || !view_ok(L.v, Hkv, kv_rows))))
    return VSA_ERR_UNSUPPORTED;
  DenseParams p;
  memset(&p, 0, sizeof(p));
  p.out = static_cast<__nv_bfloat16*>(out);
  p.out_st = to3(L.out);
  p.lse = lse;
  p.lse_seq = q_rows;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.group = Hq / Hkv;
  p.causal = causal ? 1 : 0;
  p.scale_log2 = resolve_scale(scale, D) * kLog2e;
  p.status = device_status_ptr();
  if (!p.status) return VSA_ERR_CUDA;
  const DenseTensors t{q, k, v, to3(L.q), to3(L.k), to3(L.v), q_rows, keys ? kv_rows : 0};
  const DenseBatch b{cu_seqlens_q, cu_seqlens_kv, n_seqs};
  return launch_dense_fwd(p, t, b, D, static_cast<cudaStream_t>(stream));
}

size_t dense_attn_varlen_backward_workspace_size(const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_kv,
                                                 int n_seqs, int Hq, int Hkv, int D, int64_t q_rows,
                                                 int64_t kv_rows, int causal) {
  if (check_dense(n_seqs, cu_seqlens_q, cu_seqlens_kv, Hq, Hkv, D, q_rows, kv_rows, 0.f) != VSA_OK) return 0;
  return dense_bwd_workspace(DenseBatch{cu_seqlens_q, cu_seqlens_kv, n_seqs}, Hq, Hkv, D, q_rows, causal != 0);
}

int dense_attn_varlen_backward(const void* q, const void* k, const void* v, const void* out, const void* dout,
                               const float* lse, const vsa_dense_layout* layout, const int32_t* cu_seqlens_q,
                               const int32_t* cu_seqlens_kv, int n_seqs, int Hq, int Hkv, int D,
                               int64_t q_rows, int64_t kv_rows, int causal, float scale, void* dq, void* dk,
                               void* dv, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_dense(n_seqs, cu_seqlens_q, cu_seqlens_kv, Hq, Hkv, D, q_rows, kv_rows, scale);
  if (rc != VSA_OK) return rc;
  const bool rows = cu_seqlens_q[n_seqs] > 0, keys = cu_seqlens_kv[n_seqs] > 0;
  if (!rows && !keys) return VSA_OK;
  const void* per_row[] = {q, out, dout, dq};
  const void* per_key[] = {k, v, dk, dv};
  for (int i = 0; i < 4; ++i)
    if ((rows && (!per_row[i] || !aligned16(per_row[i]))) || (keys && (!per_key[i] || !aligned16(per_key[i]))))
      return VSA_ERR_INVALID_ARG;
  if (rows && !lse) return VSA_ERR_INVALID_ARG;
  vsa_dense_layout L;
  if (layout) L = *layout;
  else contiguous_layout(&L, q_rows, kv_rows, D);
  if ((rows && (!view_ok(L.q, Hq, q_rows) || !view_ok(L.out, Hq, q_rows) || !view_ok(L.dout, Hq, q_rows) ||
                !view_ok(L.dq, Hq, q_rows))) ||
      (keys && (!view_ok(L.k, Hkv, kv_rows) || !view_ok(L.v, Hkv, kv_rows) || !view_ok(L.dk, Hkv, kv_rows) ||
                !view_ok(L.dv, Hkv, kv_rows))))
    return VSA_ERR_UNSUPPORTED;
  if (rows && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
               workspace_bytes < dense_bwd_workspace(DenseBatch{cu_seqlens_q, cu_seqlens_kv, n_seqs}, Hq, Hkv, D,
                                                     q_rows, causal != 0)))
    return VSA_ERR_WORKSPACE;
  DenseBwdParams p;
  memset(&p, 0, sizeof(p));
  p.dq = static_cast<__nv_bfloat16*>(dq);
  p.dk = static_cast<__nv_bfloat16*>(dk);
  p.dv = static_cast<__nv_bfloat16*>(dv);
  p.dq_st = to3(L.dq);
  p.dk_st = to3(L.dk);
  p.dv_st = to3(L.dv);
  p.lse = lse;
  p.delta = static_cast<float*>(workspace);
  p.lse_seq = q_rows;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.group = Hq / Hkv;
  p.causal = causal ? 1 : 0;
  p.scale = resolve_scale(scale, D);
  p.scale_log2 = p.scale * kLog2e;
  p.status = device_status_ptr();
  if (!p.status) return VSA_ERR_CUDA;
  const DenseTensors t{q, k, v, to3(L.q), to3(L.k), to3(L.v), rows ? q_rows : 0, keys ? kv_rows : 0};
  const DenseBatch b{cu_seqlens_q, cu_seqlens_kv, n_seqs};
  return launch_dense_bwd(p, t, out, to3(L.out), dout, to3(L.dout), b, D, static_cast<cudaStream_t>(stream));
}

size_t shared_prefix_attn_workspace_size(int B, int Hq, int Hkv, int T, int D, int64_t prefix_len,
                                         int64_t suffix_cap) {
  PrefixParams p;
  memset(&p, 0, sizeof(p));
  if (check_prefix(&p, B, Hq, Hkv, T, D, prefix_len, suffix_cap) != VSA_OK) return 0;
  return prefix_workspace(&p, D, nullptr);
}

int shared_prefix_attn(const void* q, const void* k_prefix, const void* v_prefix, const void* k_suffix,
                       const void* v_suffix, const int32_t* suffix_lens, const vsa_prefix_layout* layout,
                       int B, int Hq, int Hkv, int T, int D, int64_t prefix_len, int64_t suffix_cap,
                       float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                       void* stream) {
  PrefixParams p;
  memset(&p, 0, sizeof(p));
  const int rc = check_prefix(&p, B, Hq, Hkv, T, D, prefix_len, suffix_cap);
  if (rc != VSA_OK) return rc;
  if (B == 0 || T == 0) return VSA_OK;  // no rows
  const bool pfx = prefix_len > 0, sfx = suffix_cap > 0;
  if (!q || !out || !suffix_lens || !(scale == scale) || (pfx && (!k_prefix || !v_prefix)) ||
      (sfx && (!k_suffix || !v_suffix)))
    return VSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || (pfx && (!aligned16(k_prefix) || !aligned16(v_prefix))) ||
      (sfx && (!aligned16(k_suffix) || !aligned16(v_suffix))) ||
      (reinterpret_cast<uintptr_t>(suffix_lens) & 3u))
    return VSA_ERR_INVALID_ARG;
  vsa_prefix_layout L;
  if (layout) {
    L = *layout;
  } else {
    L.q = L.out = vsa_strides{(int64_t)Hq * T * D, (int64_t)T * D, D};
    L.k_prefix = L.v_prefix = vsa_strides{0, prefix_len * D, D};
    L.k_suffix = L.v_suffix = vsa_strides{Hkv * suffix_cap * D, suffix_cap * D, D};
  }
  if (!view4_ok(L.q, B, Hq, T) || !view4_ok(L.out, B, Hq, T) ||
      (pfx && (!view_ok(L.k_prefix, Hkv, prefix_len) || !view_ok(L.v_prefix, Hkv, prefix_len))) ||
      (sfx && (!view4_ok(L.k_suffix, B, Hkv, suffix_cap) || !view4_ok(L.v_suffix, B, Hkv, suffix_cap))))
    return VSA_ERR_UNSUPPORTED;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
      workspace_bytes < prefix_workspace(&p, D, workspace))
    return VSA_ERR_WORKSPACE;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.q_st = to3(L.q);
  p.out_st = to3(L.out);
  p.lse = lse;
  p.lens = suffix_lens;
  p.scale_log2 = resolve_scale(scale, D) * kLog2e;
  p.status = device_status_ptr();
  if (!p.status) return VSA_ERR_CUDA;
  const PrefixTensors t{k_prefix, v_prefix, k_suffix, v_suffix, to3(L.k_prefix), to3(L.v_prefix),
                        to3(L.k_suffix), to3(L.v_suffix)};
  return launch_prefix(p, t, D, static_cast<cudaStream_t>(stream));
}

}  // extern "C"

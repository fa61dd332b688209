// Shared by the operators on a key/value cache (tree decode, key weights,
// eviction): the drafted tokens' visibility rule and the host-side checks.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "mfa.h"
#include "mfa_internal.h"

namespace mfa {

// Sequence length of batch b, clamped to the cache.
__device__ __forceinline__ int cache_len(const int32_t* lens, int b, int N) {
  const int n = __ldg(lens + b);
  return n < 0 ? 0 : (n > N ? N : n);
}

// The parent of node t (par: the batch's parents), with everything that ends
// the way up as -1: the root, an entry outside [-2, t), a padding row.
__device__ __forceinline__ int tree_up(const int32_t* par, int t) {
  const int p = par[t];
  return (p < 0 || p >= t) ? -1 : (par[p] == -2 ? -1 : p);
}

// Whether row t sees node n's key (n == t: its own). parents NULL: a chain.
__device__ __forceinline__ bool tree_sees(const int32_t* par, int t, int n) {
  if (par == nullptr) return n <= t;
  if (n > t || par[t] == -2) return false;
  int a = t;
  while (a > n) a = tree_up(par, a);
  return a == n;
}

// The error bits of node t of batch b.
__device__ __forceinline__ uint32_t draft_errors(const int32_t* lens, const int32_t* parents, int b, int t, int T, int N) {
  const int n = __ldg(lens + b);
  bool bad = n < 0 || n > N - T;
  if (parents != nullptr) {
    const int32_t* par = parents + static_cast<int64_t>(b) * T;
    const int p = par[t];
    bad |= p < -2 || p >= t || (p >= 0 && p < t && par[p] == -2);
  }
  return bad ? MFA_DEVERR_BOUNDS : 0u;
}

// ---- host ----

// A [B, H, N, D] bf16 tensor as these operators take it: D contiguous, the
// other strides and the address on 16 bytes (the kernels' wide and TMA loads).
inline mfa_status check_cache_tensor(const mfa_tensor* t) {
  if (!t) return MFA_ERR_INVALID_ARG;
  if (t->B < 0 || t->H <= 0 || t->N < 0 || t->D <= 0) return MFA_ERR_INVALID_ARG;
  if (!t->data && t->B > 0 && t->N > 0) return MFA_ERR_INVALID_ARG;
  if (t->dtype != MFA_BF16) return MFA_ERR_UNSUPPORTED;
  if (t->stride[3] != 1) return MFA_ERR_UNSUPPORTED;
  for (int a = 0; a < 3; ++a)
    if (t->stride[a] <= 0 || (t->stride[a] * 2) % 16 != 0) return MFA_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(t->data) % 16 != 0) return MFA_ERR_UNSUPPORTED;
  return MFA_OK;
}

// The checks mfa_tree_decode and mfa_key_weights share (q and the cache k
// already checked one by one). *empty: nothing to do.
inline mfa_status check_draft(const mfa_tensor* q, const mfa_tensor* k, const int32_t* lens, const int32_t* parents,
                              const float* lse, const uint32_t* dev_err, bool* empty) {
  *empty = q->B == 0 || q->N == 0;
  if (!dev_err) return MFA_ERR_INVALID_ARG;
  if (!*empty && (!lens || !lse)) return MFA_ERR_INVALID_ARG;
  if (k->B != q->B || k->D != q->D || q->H % k->H != 0) return MFA_ERR_SHAPE_MISMATCH;
  if (q->D != 64 && q->D != 128 && q->D != 256) return MFA_ERR_UNSUPPORTED;
  if (parents && q->N > MFA_TREE_MAX_NODES) return MFA_ERR_UNSUPPORTED;
  if (k->N == 0 || k->N >= (int64_t(1) << 30) || q->N >= (int64_t(1) << 24) || q->H > 65535 || q->B > 65535)
    return MFA_ERR_UNSUPPORTED;
  if (q->B * q->H * q->N >= (int64_t(1) << 31)) return MFA_ERR_UNSUPPORTED;
  return MFA_OK;
}

}  // namespace mfa

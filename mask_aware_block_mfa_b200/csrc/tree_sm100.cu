// mfa_tree_decode: attention of a tree of drafted tokens over a cache.
//
// out[b, h, t] = sum_j p_j v_j with p = softmax over the keys j the row sees of
// q . k_j / sqrt(D): every key before lens[b], and of the drafted ones behind
// it node t itself and its ancestors.
#include <cmath>
#include <cuda_bf16.h>

#include "cache.cuh"
#include "mfa_device.cuh"

namespace mfa {
namespace {

struct TreeParams {
  int32_t B, Hq, G, T, N;
  float scale_log2;
  const __nv_bfloat16 *q, *k, *v;
  int64_t qs[3], ks[3], vs[3], os[3];
  const int32_t *lens, *parents;
  __nv_bfloat16* out;
  float* lse;
  uint32_t* err;
};

constexpr int kWarps = 8;

// One block per query row. A warp takes every eighth key: its lanes hold D / 32
// elements each, the dot product is a shuffle sum, and the softmax's running
// maximum, sum and output are kept per warp and merged at the end.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) mfa_tree_kernel(const TreeParams p) {
  constexpr int E = D / 32;
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int len = cache_len(p.lens, b, p.N);
  const int end = min(len + p.T, p.N);
  const int32_t* par = p.parents ? p.parents + static_cast<int64_t>(b) * p.T : nullptr;
  if (h == 0 && threadIdx.x == 0) {
    const uint32_t e = draft_errors(p.lens, p.parents, b, t, p.T, p.N);
    if (e) atomicOr(p.err, e);
  }
  const __nv_bfloat16* qr = p.q + b * p.qs[0] + h * p.qs[1] + t * p.qs[2] + lane * E;
  const __nv_bfloat16* kb = p.k + b * p.ks[0] + (h / p.G) * p.ks[1] + lane * E;
  const __nv_bfloat16* vb = p.v + b * p.vs[0] + (h / p.G) * p.vs[1] + lane * E;
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(qr[e]);
    o[e] = 0.f;
  }
  const bool dead = par != nullptr && par[t] == -2;
  for (int j = warp; j < end && !dead; j += kWarps) {
    if (j >= len && !tree_sees(par, t, j - len)) continue;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], __bfloat162float(kb[j * p.ks[2] + e]), s);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    s *= p.scale_log2;
    const float mn = fmaxf(m, s);
    const float a = m == -INFINITY ? 0.f : exp2f(m - mn), x = s == -INFINITY ? 0.f : exp2f(s - mn);
    m = mn;
    l = l * a + x;
    bool finite = true;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float y = __bfloat162float(vb[j * p.vs[2] + e]);
      finite &= isfinite(y);
      o[e] = o[e] * a + x * y;
    }
    // A drafted key with a value that is not finite: NaN in every column.
    if (j >= len && !__all_sync(0xffffffffu, finite)) {
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = NAN;
    }
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
  for (int w = 0; w < kWarps; ++w) L += sm[w] == -INFINITY ? sl[w] : sl[w] * exp2f(sm[w] - M);  // no maximum: 0, or NaN
  for (int d = threadIdx.x; d < D; d += kWarps * 32) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x += sm[w] == -INFINITY ? so[w][d] : so[w][d] * exp2f(sm[w] - M);
    p.out[b * p.os[0] + h * p.os[1] + t * p.os[2] + d] = __float2bfloat16_rn(L == 0.f ? 0.f : x / L);
  }
  if (threadIdx.x == 0)
    p.lse[(static_cast<int64_t>(b) * p.Hq + h) * p.T + t] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
}

}  // namespace
}  // namespace mfa

extern "C" size_t mfa_tree_decode_workspace_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t T, int32_t D) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || T < 0 || Hq % Hkv || (D != 64 && D != 128 && D != 256)) return 0;
  return 256;
}

extern "C" mfa_status mfa_tree_decode(const mfa_tensor* q, const mfa_tensor* k, const mfa_tensor* v,
                                      const int32_t* lens, const int32_t* parents, const mfa_tensor* out, float* lse,
                                      void* workspace, size_t workspace_bytes, uint32_t* dev_err, void* stream) {
  using namespace mfa;
  mfa_status st;
  if ((st = check_cache_tensor(q)) != MFA_OK || (st = check_cache_tensor(k)) != MFA_OK ||
      (st = check_cache_tensor(v)) != MFA_OK || (st = check_cache_tensor(out)) != MFA_OK)
    return st;
  bool empty;
  if ((st = check_draft(q, k, lens, parents, lse, dev_err, &empty)) != MFA_OK) return st;
  if (v->B != k->B || v->H != k->H || v->N != k->N || v->D != k->D) return MFA_ERR_SHAPE_MISMATCH;
  if (out->B != q->B || out->H != q->H || out->N != q->N || out->D != q->D) return MFA_ERR_SHAPE_MISMATCH;
  if (empty) return MFA_OK;
  const size_t need = mfa_tree_decode_workspace_bytes(static_cast<int32_t>(q->B), static_cast<int32_t>(q->H),
                                                      static_cast<int32_t>(k->H), static_cast<int32_t>(q->N),
                                                      static_cast<int32_t>(q->D));
  if (!workspace || workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
    return MFA_ERR_INVALID_ARG;
  TreeParams p;
  p.B = static_cast<int32_t>(q->B); p.Hq = static_cast<int32_t>(q->H); p.G = static_cast<int32_t>(q->H / k->H);
  p.T = static_cast<int32_t>(q->N); p.N = static_cast<int32_t>(k->N);
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(q->D)));
  p.q = static_cast<const __nv_bfloat16*>(q->data);
  p.k = static_cast<const __nv_bfloat16*>(k->data);
  p.v = static_cast<const __nv_bfloat16*>(v->data);
  for (int a = 0; a < 3; ++a) {
    p.qs[a] = q->stride[a]; p.ks[a] = k->stride[a]; p.vs[a] = v->stride[a]; p.os[a] = out->stride[a];
  }
  p.lens = lens; p.parents = parents;
  p.out = static_cast<__nv_bfloat16*>(out->data); p.lse = lse; p.err = dev_err;
  const dim3 grid(p.T, p.Hq, p.B);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (q->D == 64) mfa_tree_kernel<64><<<grid, kWarps * 32, 0, s>>>(p);
  else if (q->D == 128) mfa_tree_kernel<128><<<grid, kWarps * 32, 0, s>>>(p);
  else mfa_tree_kernel<256><<<grid, kWarps * 32, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? MFA_OK : MFA_ERR_CUDA;
}

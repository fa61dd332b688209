// mfa_key_weights: the attention weight every cached key got from a call's
// rows, w[b, g, j] = decay * w_in + sum over heads h of group g and rows t that
// see j of row_scale[t] * exp(q_ht . k_j / sqrt(D) - lse_ht).
#include <cmath>
#include <cuda_bf16.h>

#include "cache.cuh"
#include "mfa_device.cuh"

namespace mfa {
namespace {

struct KeyWeightParams {
  int32_t B, Hq, Hkv, G, T, N;
  float scale_log2, decay;
  const __nv_bfloat16 *q, *k;
  int64_t qs[3], ks[3];
  const float *lse, *row_scale, *w_in;
  const int32_t *lens, *parents;
  float* w_out;
  uint32_t* err;
};

constexpr int kWarps = 8;

// A warp per key; its lanes hold D / 32 elements of it each.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) mfa_key_weights_kernel(const KeyWeightParams p) {
  constexpr int E = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = blockIdx.y, b = blockIdx.z;
  const int len = cache_len(p.lens, b, p.N);
  const int end = min(len + p.T, p.N);
  const int32_t* par = p.parents ? p.parents + static_cast<int64_t>(b) * p.T : nullptr;
  if (blockIdx.x == 0 && g == 0) {
    for (int t = threadIdx.x; t < p.T; t += kWarps * 32) {
      const uint32_t e = draft_errors(p.lens, p.parents, b, t, p.T, p.N);
      if (e) atomicOr(p.err, e);
    }
  }
  for (int j = blockIdx.x * kWarps + warp; j < end; j += gridDim.x * kWarps) {
    float k[E], acc = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) k[e] = __bfloat162float(p.k[b * p.ks[0] + g * p.ks[1] + j * p.ks[2] + lane * E + e]);
    for (int t = 0; t < p.T; ++t) {
      const float r = p.row_scale ? p.row_scale[static_cast<int64_t>(b) * p.T + t] : 1.f;
      if (r == 0.f || (par && par[t] == -2) || (j >= len && !tree_sees(par, t, j - len))) continue;
      for (int h = g * p.G; h < (g + 1) * p.G; ++h) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e)
          s = fmaf(k[e], __bfloat162float(p.q[b * p.qs[0] + h * p.qs[1] + t * p.qs[2] + lane * E + e]), s);
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
        const float lse = p.lse[(static_cast<int64_t>(b) * p.Hq + h) * p.T + t];
        if (lse != -INFINITY) acc = fmaf(r, exp2f(s * p.scale_log2 - lse * 1.44269504f), acc);
      }
    }
    if (lane == 0) {
      const int64_t at = (static_cast<int64_t>(b) * p.Hkv + g) * p.N + j;
      p.w_out[at] = p.decay != 0.f && p.w_in ? fmaf(p.decay, p.w_in[at], acc) : acc;
    }
  }
}

}  // namespace
}  // namespace mfa

extern "C" mfa_status mfa_key_weights(const mfa_tensor* q, const mfa_tensor* k, const float* lse, const int32_t* lens,
                                      const int32_t* parents, const float* row_scale, const float* weights_in,
                                      float decay, float* weights_out, uint32_t* dev_err, void* stream) {
  using namespace mfa;
  mfa_status st;
  if ((st = check_cache_tensor(q)) != MFA_OK || (st = check_cache_tensor(k)) != MFA_OK) return st;
  bool empty;
  if ((st = check_draft(q, k, lens, parents, lse, dev_err, &empty)) != MFA_OK) return st;
  if (q->N == 0) return MFA_ERR_UNSUPPORTED;
  if (empty) return MFA_OK;
  if (!weights_out) return MFA_ERR_INVALID_ARG;
  KeyWeightParams p;
  p.B = static_cast<int32_t>(q->B); p.Hq = static_cast<int32_t>(q->H); p.Hkv = static_cast<int32_t>(k->H);
  p.G = static_cast<int32_t>(q->H / k->H); p.T = static_cast<int32_t>(q->N); p.N = static_cast<int32_t>(k->N);
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(q->D)));
  p.decay = decay;
  p.q = static_cast<const __nv_bfloat16*>(q->data);
  p.k = static_cast<const __nv_bfloat16*>(k->data);
  for (int a = 0; a < 3; ++a) {
    p.qs[a] = q->stride[a]; p.ks[a] = k->stride[a];
  }
  p.lse = lse; p.row_scale = row_scale; p.w_in = weights_in; p.w_out = weights_out;
  p.lens = lens; p.parents = parents; p.err = dev_err;
  const int64_t blocks = cdiv64(p.N, kWarps);
  const dim3 grid(static_cast<unsigned>(blocks < 256 ? blocks : 256), p.Hkv, p.B);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (q->D == 64) mfa_key_weights_kernel<64><<<grid, kWarps * 32, 0, s>>>(p);
  else if (q->D == 128) mfa_key_weights_kernel<128><<<grid, kWarps * 32, 0, s>>>(p);
  else mfa_key_weights_kernel<256><<<grid, kWarps * 32, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? MFA_OK : MFA_ERR_CUDA;
}

// Eviction from a key/value cache by accumulated attention weight:
// mfa_evict_select chooses the keys to keep, mfa_cache_compact moves the rows.
#include <cuda_bf16.h>

#include "cache.cuh"

namespace mfa {
namespace {

// ---------------------------------------------------------------------------
// Selection. The k largest of m weights by radix selection: a weight becomes an
// unsigned key of the same order, and four passes of eight bits, from the
// top, narrow down the k-th largest key: each counts the keys that agree with
// the bits found so far by their next eight bits. Keys above the k-th are
// kept, and of those equal to it the first ones by index.
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;

struct SelectParams {
  const float* weights;
  const int32_t* lens;
  int32_t Hkv, N, budget, recent;
  int32_t *keep, *new_lens;
  uint32_t* err;
};

// Ordered key of a weight; NaN as -inf, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float x) {
  uint32_t u = __float_as_uint(x);
  if (x != x) u = 0xff800000u;
  if (x == 0.f) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kSelThreads) mfa_select_kernel(const SelectParams p) {
  __shared__ int hist[256];
  __shared__ int s_bin, s_left;
  __shared__ int s_gt[kSelWarps], s_eq[kSelWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = blockIdx.x, b = blockIdx.y;
  const int raw = __ldg(p.lens + b);
  const int n = cache_len(p.lens, b, p.N);
  const int kept = min(n, p.budget);
  const int64_t row = static_cast<int64_t>(b) * p.Hkv + g;
  int32_t* keep = p.keep + row * p.budget;
  if (g == 0 && threadIdx.x == 0) {
    p.new_lens[b] = kept;
    if (raw != n) atomicOr(p.err, MFA_DEVERR_BOUNDS);
  }
  for (int t = kept + threadIdx.x; t < p.budget; t += kSelThreads) keep[t] = -1;
  if (n <= p.budget) {
    for (int t = threadIdx.x; t < n; t += kSelThreads) keep[t] = t;
    return;
  }
  const int m = n - p.recent, k = p.budget - p.recent;  // the k largest of the first m; m > k
  for (int t = threadIdx.x; t < p.recent; t += kSelThreads) keep[k + t] = m + t;
  if (k == 0) return;
  const float* w = p.weights + row * p.N;
  uint32_t prefix = 0;
  int left = k;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (threadIdx.x < 256) hist[threadIdx.x] = 0;
    __syncthreads();
    for (int j = threadIdx.x; j < m; j += kSelThreads) {
      const uint32_t key = order_key(__ldg(w + j));
      if (shift == 24 || (key >> (shift + 8)) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int bin = 255, rest = left;
      while (hist[bin] < rest) rest -= hist[bin--];
      s_bin = bin;
      s_left = rest;
    }
    __syncthreads();
    prefix = (prefix << 8) | static_cast<uint32_t>(s_bin);
    left = s_left;
  }
  // prefix is the k-th largest key, `left` of its equals are kept.
  const int seg = ((m + kSelThreads - 1) / kSelThreads) * 32;
  const int j0 = warp * seg, j1 = min(m, j0 + seg);
  int gt = 0, eq = 0;
  for (int j = j0 + lane; j < j1; j += 32) {
    const uint32_t key = order_key(__ldg(w + j));
    gt += key > prefix;
    eq += key == prefix;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    s_gt[warp] = gt;
    s_eq[warp] = eq;
  }
  __syncthreads();
  gt = eq = 0;
  for (int x = 0; x < warp; ++x) {
    gt += s_gt[x];
    eq += s_eq[x];
  }
  for (int base = j0; base < j1; base += 32) {
    const int j = base + lane;
    const uint32_t key = j < j1 ? order_key(__ldg(w + j)) : 0u;
    const bool is_gt = j < j1 && key > prefix, is_eq = j < j1 && key == prefix;
    const unsigned below = (1u << lane) - 1u;
    const unsigned bg = __ballot_sync(0xffffffffu, is_gt), be = __ballot_sync(0xffffffffu, is_eq);
    const int eb = eq + __popc(be & below);
    if (is_gt || (is_eq && eb < left)) keep[gt + __popc(bg & below) + min(eb, left)] = j;
    gt += __popc(bg);
    eq += __popc(be);
  }
}

// ---------------------------------------------------------------------------
// Moving rows together. In place the destination rows are the sources of
// earlier or the same entries only (idx[t] >= t), so a block that takes the
// entries in order, a chunk at a time, and loads a whole chunk before it
// stores any of it, reads every row before it is overwritten. Blocks share
// nothing: each moves its own slice of a head's columns.
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 256;
constexpr int kSlice = 4;                            // 16-byte units of a row per block
constexpr int kMoveRows = kMoveThreads / kSlice;     // entries per chunk

struct CompactParams {
  int32_t B, Hkv, idx_heads, n_idx, units;  // units: 16-byte units of a row
  int64_t N, N_out;
  bool in_place;
  const uint4 *k, *v;
  uint4 *k_out, *v_out;
  int64_t ks[3], vs[3], kos[3], vos[3];  // strides in 16-byte units
  const float* w;
  float* w_out;
  const int32_t *start, *idx, *count, *zero_end;
  uint32_t* err;
};

__global__ void __launch_bounds__(kMoveThreads) mfa_compact_kernel(const CompactParams p) {
  const int g = blockIdx.y, b = blockIdx.z;
  const int slices = (p.units + kSlice - 1) / kSlice;
  const int64_t s = p.start ? __ldg(p.start + b) : 0;
  const int count = min(max(__ldg(p.count + b), 0), p.n_idx);
  const int32_t* idx = p.idx + (static_cast<int64_t>(b) * p.idx_heads + (p.idx_heads == 1 ? 0 : g)) * p.n_idx;
  // The source row of entry t, or -1 when it moves nothing.
  auto source = [&](int t, bool report) -> int64_t {
    const int64_t x = __ldg(idx + t);
    const bool bad = x < 0 || s + x < 0 || s + x >= p.N || s + t < 0 || s + t >= p.N_out || (p.in_place && x < t);
    if (bad && report) atomicOr(p.err, MFA_DEVERR_SEL);
    return bad || (p.in_place && x == t) ? -1 : s + x;
  };
  if (blockIdx.x < 2 * slices) {
    const bool isv = blockIdx.x >= slices;
    const int slice = blockIdx.x - (isv ? slices : 0);
    const int u = slice * kSlice + threadIdx.x % kSlice;
    const int64_t* si = isv ? p.vs : p.ks;
    const int64_t* so = isv ? p.vos : p.kos;
    const uint4* src = (isv ? p.v : p.k) + b * si[0] + g * si[1] + u;
    uint4* dst = (isv ? p.v_out : p.k_out) + b * so[0] + g * so[1] + u;
    for (int base = 0; base < count; base += kMoveRows) {
      const int t = base + threadIdx.x / kSlice;
      int64_t r = -1;
      uint4 x;
      if (t < count && u < p.units) {
        r = source(t, blockIdx.x == 0);
        if (r >= 0) x = src[r * si[2]];
      }
      __syncthreads();
      if (r >= 0) dst[(s + t) * so[2]] = x;
    }
  } else if (p.w_out) {
    const float* src = p.w + (static_cast<int64_t>(b) * p.Hkv + g) * p.N;
    float* dst = p.w_out + (static_cast<int64_t>(b) * p.Hkv + g) * p.N_out;
    for (int base = 0; base < count; base += kMoveThreads) {
      const int t = base + threadIdx.x;
      int64_t r = -1;
      float x = 0.f;
      if (t < count) {
        r = source(t, false);
        if (r >= 0) x = src[r];
      }
      __syncthreads();
      if (r >= 0) dst[s + t] = x;
    }
    __syncthreads();
    if (p.zero_end) {
      const int64_t z = min(static_cast<int64_t>(__ldg(p.zero_end + b)), p.N_out);
      for (int64_t j = max(s + count, int64_t(0)) + threadIdx.x; j < z; j += kMoveThreads) dst[j] = 0.f;
    }
  }
}

// The bytes of a [B, H, N, ...] tensor, first to last, as an address range.
struct Range {
  uintptr_t lo, hi;
};
Range tensor_range(const mfa_tensor* t) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(t->data);
  const int64_t last = (t->B - 1) * t->stride[0] + (t->H - 1) * t->stride[1] + (t->N - 1) * t->stride[2] + t->D;
  return {lo, lo + static_cast<uintptr_t>(last) * 2};
}
bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }
bool same_tensor(const mfa_tensor* a, const mfa_tensor* b) {
  return a->data == b->data && a->N == b->N && a->stride[0] == b->stride[0] && a->stride[1] == b->stride[1] &&
         a->stride[2] == b->stride[2];
}

}  // namespace
}  // namespace mfa

extern "C" mfa_status mfa_evict_select(const float* weights, const int32_t* lens, int32_t B, int32_t Hkv, int32_t N,
                                       int32_t budget, int32_t recent, int32_t* keep, int32_t* new_lens,
                                       uint32_t* dev_err, void* stream) {
  using namespace mfa;
  if (B < 0 || Hkv <= 0 || N <= 0 || budget <= 0 || recent < 0 || recent > budget || !dev_err)
    return MFA_ERR_INVALID_ARG;
  if (B == 0) return MFA_OK;
  if (!weights || !lens || !keep || !new_lens || lens == new_lens) return MFA_ERR_INVALID_ARG;
  if (N >= (1 << 30) || budget >= (1 << 30) || Hkv > 65535 || B > 65535 || static_cast<int64_t>(B) * Hkv > (1 << 24))
    return MFA_ERR_UNSUPPORTED;
  SelectParams p{weights, lens, Hkv, N, budget, recent, keep, new_lens, dev_err};
  mfa_select_kernel<<<dim3(Hkv, B), kSelThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? MFA_OK : MFA_ERR_CUDA;
}

extern "C" mfa_status mfa_cache_compact(const mfa_tensor* k, const mfa_tensor* v, const float* weights,
                                        const int32_t* start, const int32_t* idx, int32_t idx_heads, int32_t n_idx,
                                        const int32_t* count, const int32_t* zero_end, const mfa_tensor* k_out,
                                        const mfa_tensor* v_out, float* weights_out, uint32_t* dev_err, void* stream) {
  using namespace mfa;
  mfa_status st;
  if ((st = check_cache_tensor(k)) != MFA_OK || (st = check_cache_tensor(v)) != MFA_OK ||
      (st = check_cache_tensor(k_out)) != MFA_OK || (st = check_cache_tensor(v_out)) != MFA_OK)
    return st;
  if (!dev_err || n_idx < 0 || idx_heads <= 0 || (weights == nullptr) != (weights_out == nullptr))
    return MFA_ERR_INVALID_ARG;
  if (zero_end && !weights) return MFA_ERR_INVALID_ARG;
  if (v->B != k->B || v->H != k->H || v->N != k->N || v->D != k->D) return MFA_ERR_SHAPE_MISMATCH;
  for (const mfa_tensor* o : {k_out, v_out})
    if (o->B != k->B || o->H != k->H || o->D != k->D || o->N != k_out->N) return MFA_ERR_SHAPE_MISMATCH;
  if (idx_heads != 1 && idx_heads != k->H) return MFA_ERR_SHAPE_MISMATCH;
  if (k->D % 8 != 0 || k->D > 512) return MFA_ERR_UNSUPPORTED;
  if (k->B > 65535 || k->H > 65535 || k->N >= (int64_t(1) << 30) || k_out->N >= (int64_t(1) << 30))
    return MFA_ERR_UNSUPPORTED;
  if (k->B == 0 || k->N == 0 || k_out->N == 0) return MFA_OK;
  if (!count || (!idx && n_idx > 0)) return MFA_ERR_INVALID_ARG;
  const bool in_place = same_tensor(k, k_out);
  if (in_place != same_tensor(v, v_out)) return MFA_ERR_INVALID_ARG;
  const Range rk = tensor_range(k), rv = tensor_range(v), ro = tensor_range(k_out), rp = tensor_range(v_out);
  if (in_place) {
    // Interleaved caches (K and V of a token side by side) are in place: they
    // overlap as ranges but share no row; the same base address does not.
    if (k->data == v->data) return MFA_ERR_INVALID_ARG;
  } else if (overlap(rk, ro) || overlap(rk, rp) || overlap(rv, ro) || overlap(rv, rp) || k_out->data == v_out->data) {
    return MFA_ERR_INVALID_ARG;
  }
  if (weights) {
    const uintptr_t w = reinterpret_cast<uintptr_t>(weights), o = reinterpret_cast<uintptr_t>(weights_out);
    const Range rw{w, w + static_cast<uintptr_t>(k->B * k->H * k->N) * 4};
    const Range rx{o, o + static_cast<uintptr_t>(k->B * k->H * k_out->N) * 4};
    if (in_place ? weights != weights_out : overlap(rw, rx)) return MFA_ERR_INVALID_ARG;
  }
  CompactParams p;
  p.B = static_cast<int32_t>(k->B); p.Hkv = static_cast<int32_t>(k->H); p.idx_heads = idx_heads; p.n_idx = n_idx;
  p.units = static_cast<int32_t>(k->D / 8); p.N = k->N; p.N_out = k_out->N; p.in_place = in_place;
  p.k = static_cast<const uint4*>(k->data); p.v = static_cast<const uint4*>(v->data);
  p.k_out = static_cast<uint4*>(k_out->data); p.v_out = static_cast<uint4*>(v_out->data);
  for (int a = 0; a < 3; ++a) {
    p.ks[a] = k->stride[a] / 8; p.vs[a] = v->stride[a] / 8;
    p.kos[a] = k_out->stride[a] / 8; p.vos[a] = v_out->stride[a] / 8;
  }
  p.w = weights; p.w_out = weights_out;
  p.start = start; p.idx = idx; p.count = count; p.zero_end = zero_end; p.err = dev_err;
  const int slices = (p.units + kSlice - 1) / kSlice;
  const dim3 grid(2 * slices + (weights ? 1 : 0), p.Hkv, p.B);
  mfa_compact_kernel<<<grid, kMoveThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? MFA_OK : MFA_ERR_CUDA;
}

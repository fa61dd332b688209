// Shared by the operators on a key/value cache (tree decode, key weights,
// eviction): the drafted tokens' visibility rule and the host-side checks.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "mfa.h"
#include "mfa_device.cuh"
#include "mfa_internal.h"

namespace mfa {

// Sequence length of batch b, clamped to the cache.
__device__ __forceinline__ int cache_len(const int32_t* lens, int b, int N) {
  const int n = lens[b];
  return n < 0 ? 0 : (n > N ? N : n);
}

// The parent of node t (par: the batch's parents), with everything that ends
// the way up as -1: the root, an entry outside [-2, t), a padding row.
template <typename T>
__device__ __forceinline__ int tree_up(const T* par, int t) {
  const int p = par[t];
  return (p < 0 || p >= t) ? -1 : (par[p] == -2 ? -1 : p);
}

// Division of numbers below 2^31 by a divisor known on the host: with
// 2^(shift - 1) < d <= 2^shift and mul = ceil(2^(31 + shift) / d), n mul / 2^(31 + shift)
// exceeds n / d by less than n / 2^31 / d < 1 / d.
struct FastDiv {
  uint32_t mul, shift;
  __host__ void set(uint32_t d) {
    shift = 0;
    while ((uint64_t(1) << shift) < d) ++shift;
    mul = static_cast<uint32_t>(((uint64_t(1) << (31 + shift)) + d - 1) / d);
  }
  __device__ __forceinline__ int operator()(int n) const {
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * mul) >> (31 + shift));
  }
};

// Which of the X rows from `first` on (row = node * G + head) see the key of `node`, as
// bits: in a chain the rows from first + from on; in a tree by the table
// seen[T][words] of the nodes each node sees.
__device__ __forceinline__ uint32_t rows_from(int from) { return from <= 0 ? ~0u : from >= 32 ? 0u : ~0u << from; }
template <int X>
__device__ __forceinline__ uint32_t rows_seeing(const uint32_t* seen, int words, int node, int first, int G, FastDiv by_g, int T) {
  uint32_t bits = 0u;
  const uint32_t* col = seen + (node >> 5);
  const int t0 = by_g(first), t1 = min(by_g(first + X - 1), T - 1);
#pragma unroll 4
  for (int t = t0; t <= t1; ++t) {
    const uint32_t yes = (col[t * words] >> (node & 31)) & 1u;
    const int lo = max(t * G - first, 0), hi = min((t + 1) * G - first, X);  // its rows: [lo, hi)
    bits |= yes ? rows_from(lo) & ~rows_from(hi) : 0u;
  }
  return bits;
}

// The error bits of node t of batch b.
__device__ __forceinline__ uint32_t draft_errors(const int32_t* lens, const int32_t* parents, int b, int t, int T, int N) {
  const int n = lens[b];
  bool bad = n < 0 || n > N - T;
  if (parents != nullptr) {
    const int32_t* par = parents + static_cast<int64_t>(b) * T;
    const int p = par[t];
    bad |= p < -2 || p >= t || (p >= 0 && p < t && par[p] == -2);
  }
  return bad ? MFA_DEVERR_BOUNDS : 0u;
}

constexpr int kKeys = 128;           // keys per tile
constexpr int kChunk = kKeys * 128;  // bytes of 64 columns of a tile, 128-byte swizzled rows

// The line that is cut among the CTAs: the tiles of all (batch, head) pairs end
// to end, each pair's up to the key of node t_hi, with `extra` more places
// before them for what it costs to begin and end a pair.
struct Line {
  const int32_t* lens;
  int B, Hkv, N, t_hi, extra;
  __device__ __forceinline__ int len(int b) const { return cache_len(lens, b, N); }
  __device__ __forceinline__ int tiles(int n) const { return (min(n + t_hi + 1, N) + kKeys - 1) / kKeys; }
};

__device__ __forceinline__ int places_per_cta(int total, int ctas) {
  return static_cast<int>((static_cast<unsigned>(total) + ctas - 1) / ctas);
}

// Where CTA `cta` of `ctas` begins, found by each warp for itself (for up to 32 batches one
// load and two shuffle reductions, without a block barrier): the line's length, the CTA's
// first place, the batch that holds it (-1: past the end) and the length before that batch.
struct Start {
  int total, begin, before, b, len;  // len: of batch b
};
__device__ __forceinline__ Start find_start(const Line& ln, int cta, int ctas) {
  const int lane = threadIdx.x & 31;
  Start s{0, 0, 0, -1, 0};
  int keep = 0, n = 0;  // of batch `lane` of the last 32, and its length
  for (int b0 = 0; b0 < ln.B; b0 += 32) {
    n = b0 + lane < ln.B ? ln.len(b0 + lane) : 0;
    keep = b0 + lane < ln.B ? ln.tiles(n) + ln.extra : 0;
    s.total += __reduce_add_sync(0xffffffffu, keep);
  }
  s.total *= ln.Hkv;
  s.begin = cta * places_per_cta(s.total, ctas);
  int done = 0;  // of the batches before
  for (int b0 = 0; b0 < ln.B && s.b < 0; b0 += 32) {
    if (ln.B > 32) {
      n = b0 + lane < ln.B ? ln.len(b0 + lane) : 0;
      keep = b0 + lane < ln.B ? ln.tiles(n) + ln.extra : 0;
    }
    int sum = keep;
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, sum, w);
      if (lane >= w) sum += o;
    }
    const unsigned in = __ballot_sync(0xffffffffu, s.begin < done + sum * ln.Hkv);
    if (in) {
      const int l = __ffs(in) - 1;
      s.b = b0 + l < ln.B ? b0 + l : -1;
      s.len = __shfl_sync(0xffffffffu, n, l);
      s.before = done + __shfl_sync(0xffffffffu, sum - keep, l) * ln.Hkv;
    }
    done += __shfl_sync(0xffffffffu, sum, 31) * ln.Hkv;
  }
  return s;
}

// The (batch, head) pairs of a CTA's range, one after the other, with the tiles
// [t0, t1) of each.
struct Walk {
  int b, g, t0, t1, len, nt;
  int left;  // of the range not yet given out
  bool more;
  __device__ __forceinline__ Walk(const Line& ln, const Start& s, int ctas) {
    left = min(places_per_cta(s.total, ctas), s.total - s.begin);
    b = s.b;
    len = s.len;
    nt = ln.tiles(len);
    const int in = s.begin - s.before;
    g = in / (nt + ln.extra);
    more = take(ln, in - g * (nt + ln.extra)) || next(ln);
  }
  // The pair's part of the range from place v of the pair on; false when it holds no tile.
  __device__ __forceinline__ bool take(const Line& ln, int v) {
    const int v1 = min(nt + ln.extra, v + left);
    left -= v1 - v;
    t0 = max(v - ln.extra, 0);
    t1 = max(v1 - ln.extra, 0);
    return t1 > t0;
  }
  // The next pair; false at the range's end.
  __device__ __forceinline__ bool next(const Line& ln) {
    if (left <= 0) return more = false;
    if (++g == ln.Hkv) {
      g = 0;
      ++b;
      len = ln.len(b);
      nt = ln.tiles(len);
    }
    return more = take(ln, 0);  // (only the range's last pair can hold no tile)
  }
};

// D[tmem] = A B^T of 128 x N, both operands in shared memory, K-major or both MN-major.
__host__ __device__ constexpr uint32_t idesc_keys(int N, bool mn_major) {
  return idesc_bf16_f32(128, N, mn_major) | (mn_major ? 1u << 15 : 0u);
}

// Waits of a whole warp for one barrier, and for two at once (the lanes share them out: a
// wait that is over still takes about 130 cycles beside 16 busy warps).
__device__ __forceinline__ bool warp_wait(uint64_t* a, uint32_t pa, volatile int* abort) {
  return __all_sync(0xffffffffu, mbar_wait(a, pa, abort)) != 0;
}
__device__ __forceinline__ bool warp_wait2(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, volatile int* abort) {
  const bool odd = threadIdx.x & 1;
  return __all_sync(0xffffffffu, mbar_wait(odd ? b : a, odd ? pb : pa, abort)) != 0;
}

// A named barrier that tells whether x holds in any of its threads.
__device__ __forceinline__ bool vote_or(uint32_t id, uint32_t threads, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r) : "r"(x ? 1u : 0u), "r"(id), "r"(threads) : "memory");
  return r != 0;
}

// ---- host ----

// A launch that may begin while the kernel before it in the stream ends (the
// kernel waits for that one, griddepcontrol.wait, before it reads anything; what it reads then
// may have been written while it was already there, so no load is a
// non-coherent one).
template <typename... P, typename... A>
inline bool launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

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

// Whether the line's places can be counted in 32 bits (with the largest `extra`).
inline bool line_fits(const mfa_tensor* k) { return k->B * k->H * (cdiv64(k->N, kKeys) + 16) < (int64_t(1) << 30); }

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
  if (q->B * q->H * q->N >= (int64_t(1) << 30) || !line_fits(k)) return MFA_ERR_UNSUPPORTED;
  return MFA_OK;
}

// The tensor map of a cache tensor: boxes of 64 columns x 128 keys of one head.
inline bool map_keys(CUtensorMap* map, const mfa_tensor* t) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(t->D), static_cast<cuuint64_t>(t->N), static_cast<cuuint64_t>(t->H),
                        static_cast<cuuint64_t>(t->B)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(t->stride[2]) * 2, static_cast<cuuint64_t>(t->stride[1]) * 2,
                           static_cast<cuuint64_t>(t->stride[0]) * 2};
  cuuint32_t box[4] = {64, kKeys, 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, t->data, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, t->D == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace mfa

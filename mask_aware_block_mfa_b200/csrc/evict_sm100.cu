// Eviction from a key/value cache by accumulated attention weight:
// mfa_evict_select chooses the keys to keep, mfa_cache_compact moves the rows.
#include <algorithm>
#include <cuda_bf16.h>

#include "cache.cuh"

namespace mfa {
namespace {

// ---------------------------------------------------------------------------
// Selection. The k largest of m weights by radix selection: a weight becomes an
// unsigned key of the same order, and three passes of 11, 11 and 10 bits, from
// the top, narrow down the k-th largest key: each counts the keys that agree
// with the bits found so far by their next bits. Keys above the k-th are kept, and
// of those equal to it the first ones by index. (64 lists of 27,000 on average: 19 us.)
//
// One block per (batch, head) holds its keys in shared memory, so that the
// weights are read once (lists beyond kSelShared keys are read again for each
// pass; they sit in L2). A warp owns a run of keys, so that the kept rows'
// places follow from ballots and one scan over the warps. Bound: issue slots and
// the counters' atomics. Equal keys serialise those, and accumulated weights
// hold many zeros: zeros are counted in a register, and 32 keys of one bin
// by one lane. (A cluster of 2 to 8 blocks per list, each counting its share and
// reading the others' counts, measured 20 us against 12 on 15 lists of 20011: its
// three barriers and remote reads cost more than the shorter passes save.)
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kRun = 128;               // a warp's keys at a time, four per lane
constexpr int kSelShared = 48 * 1024;   // with hist, what a block may hold

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
constexpr uint32_t kZeroKey = 0x80000000u;

// SHARED: the keys in shared memory; otherwise read again for each pass.
// LIST: the kept keys' rows are put in order in shared memory too, and written from
// there side by side (64 lists of 8192 of 32768: 3 us less than scattered writes).
template <bool SHARED, bool LIST>
__global__ void __launch_bounds__(kSelThreads, 1) mfa_select_kernel(const __grid_constant__ SelectParams p) {
  __shared__ int hist[3][kBins];
  __shared__ int s_sum[kSelWarps], s_gt[kSelWarps], s_eq[kSelWarps];
  __shared__ int s_bin, s_left;
  extern __shared__ __align__(16) uint32_t s_keys[];  // the keys; with LIST the kept ones' rows behind them
  for (int i = threadIdx.x; i < 3 * kBins; i += kSelThreads) (&hist[0][0])[i] = 0;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = blockIdx.x, b = blockIdx.y;
  const int raw = p.lens[b];
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
  // A warp owns `seg` keys from j0 on; places past the list hold key 0, which no weight has.
  const int seg = (m + kSelWarps * kRun - 1) / (kSelWarps * kRun) * kRun, j0 = warp * seg;
  uint32_t* own = s_keys + j0;
  if constexpr (SHARED) {
#pragma unroll 8
    for (int i = lane; i < seg; i += 32) own[i] = j0 + i < m ? order_key(w[j0 + i]) : 0u;
  }
  __syncthreads();
  // Lane `lane`'s keys j0 + i + 4 * lane .. + 3.
  auto four = [&](int i, uint32_t (&key)[4]) {
    if constexpr (SHARED) {
      const uint4 x = *reinterpret_cast<const uint4*>(own + i + lane * 4);
      key[0] = x.x; key[1] = x.y; key[2] = x.z; key[3] = x.w;
    } else {
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int j = j0 + i + lane * 4 + y;
        key[y] = j < m ? order_key(w[j]) : 0u;
      }
    }
  };
  uint32_t prefix = 0;
  int left = k;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, above = pass == 0 ? 31 : pass == 1 ? 21 : 10;
    const uint32_t mask = pass == 2 ? 1023u : 2047u;
    const bool has_zero = pass == 0 || (kZeroKey >> above) == prefix;  // zero may be among the keys counted
    int zeros = 0;
#pragma unroll 2
    for (int i = 0; i < seg; i += kRun) {
      uint32_t key[4];
      four(i, key);
      bool in[4], any = false;
      int bin[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        in[y] = pass == 0 ? key[y] != 0u : (key[y] >> above) == prefix;
        bin[y] = (key[y] >> shift) & mask;
        any |= in[y];
      }
      if (pass > 0 && !__any_sync(0xffffffffu, any)) continue;  // few keys get past the first digit
      if (__all_sync(0xffffffffu, in[0] && in[1] && in[2] && in[3])) {
        const int first = __shfl_sync(0xffffffffu, bin[0], 0);
        if (__all_sync(0xffffffffu, bin[0] == first && bin[1] == first && bin[2] == first && bin[3] == first)) {
          if (lane == 0) atomicAdd(&hist[pass][first], kRun);
          continue;
        }
      }
      if (has_zero) {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          zeros += in[y] && key[y] == kZeroKey;
          if (in[y] && key[y] != kZeroKey) atomicAdd(&hist[pass][bin[y]], 1);
        }
      } else {
#pragma unroll
        for (int y = 0; y < 4; ++y)
          if (in[y]) atomicAdd(&hist[pass][bin[y]], 1);
      }
    }
    zeros = __reduce_add_sync(0xffffffffu, zeros);
    if (lane == 0 && zeros > 0) atomicAdd(&hist[pass][(kZeroKey >> shift) & mask], zeros);
    __syncthreads();
    // The bin that holds the left-th largest: thread t looks at bins top - 2t and top - 2t - 1.
    const int hi = static_cast<int>(kBins) - 1 - 2 * threadIdx.x;
    const int a = hist[pass][hi], c = hist[pass][hi - 1];
    int sum = a + c;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, sum, x);
      if (lane >= x) sum += o;
    }
    if (lane == 31) s_sum[warp] = sum;
    __syncthreads();
    int base = lane < warp ? s_sum[lane] : 0;
    base = __reduce_add_sync(0xffffffffu, base);
    const int before = base + sum - a - c;  // keys in higher bins
    if (before < left && before + a >= left) {
      s_bin = hi;
      s_left = left - before;
    } else if (before + a < left && before + a + c >= left) {
      s_bin = hi - 1;
      s_left = left - before - a;
    }
    __syncthreads();
    prefix = (prefix << (pass == 2 ? 10 : 11)) | static_cast<uint32_t>(s_bin);
    left = s_left;
  }
  // prefix is the k-th largest key, `left` of its equals are kept.
  int gt = 0, eq = 0;
#pragma unroll 4
  for (int i = 0; i < seg; i += kRun) {
    uint32_t key[4];
    four(i, key);
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      gt += key[y] > prefix;
      eq += key[y] == prefix;
    }
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    s_gt[warp] = gt;
    s_eq[warp] = eq;
  }
  __syncthreads();
  int32_t* list = LIST ? reinterpret_cast<int32_t*>(s_keys + seg * kSelWarps) : keep;
  gt = __reduce_add_sync(0xffffffffu, lane < warp ? s_gt[lane] : 0);
  eq = __reduce_add_sync(0xffffffffu, lane < warp ? s_eq[lane] : 0);
  // A kept key's place: the keys above the k-th before it, and the equal ones that are kept.
  const unsigned below = (1u << lane) - 1u;
#pragma unroll 2
  for (int i = 0; i < seg; i += kRun) {
    uint32_t key[4];
    four(i, key);
    int at = gt, ties = eq;
    bool tie = false;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const unsigned bg = __ballot_sync(0xffffffffu, key[y] > prefix);
      at += __popc(bg & below);
      gt += __popc(bg);
      tie |= key[y] == prefix;
    }
    if (__any_sync(0xffffffffu, tie)) {
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const unsigned be = __ballot_sync(0xffffffffu, key[y] == prefix);
        ties += __popc(be & below);
        eq += __popc(be);
      }
    }
    const int j = j0 + i + lane * 4;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const bool is_gt = key[y] > prefix, is_eq = key[y] == prefix;
      if (is_gt || (is_eq && ties < left)) list[at + min(ties, left)] = j + y;
      at += is_gt;
      ties += is_eq;
    }
  }
  if constexpr (LIST) {
    __syncthreads();
    for (int t = threadIdx.x; t < k; t += kSelThreads) keep[t] = list[t];
  }
}

// ---------------------------------------------------------------------------
// Moving rows together. Bound: HBM, every kept row read and written once (64 lists of
// 8192 of 32768 rows of 128 columns: 85 us, 6.3 TB/s).
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 256;

struct CompactParams {
  int32_t B, Hkv, idx_heads, n_idx, units;  // units: 16-byte units of a row
  int64_t N, N_out;
  const uint4 *k, *v;
  uint4 *k_out, *v_out;
  int64_t ks[3], vs[3], kos[3], vos[3];  // strides in 16-byte units
  const float* w;
  float* w_out;
  const int32_t *start, *idx, *count, *zero_end;
  uint32_t* err;
};

// One (batch, head)'s list.
struct Moves {
  int64_t s;
  int count;
  const int32_t* idx;
  __device__ __forceinline__ Moves(const CompactParams& p, int g, int b) {
    s = p.start ? p.start[b] : 0;
    count = min(max(p.count[b], 0), p.n_idx);
    idx = p.idx + (static_cast<int64_t>(b) * p.idx_heads + (p.idx_heads == 1 ? 0 : g)) * p.n_idx;
  }
  // The source row of entry t of a move into other tensors, or -1 when it moves nothing.
  __device__ __forceinline__ int64_t source(const CompactParams& p, int t) const {
    const int64_t x = idx[t];
    const bool bad = x < 0 || s + x < 0 || s + x >= p.N || s + t < 0 || s + t >= p.N_out;
    if (bad) atomicOr(p.err, MFA_DEVERR_SEL);
    return bad ? -1 : s + x;
  }
};

__device__ __forceinline__ void zero_tail(const CompactParams& p, const Moves& mv, float* dst, int b, int64_t first, int64_t step) {
  if (!p.zero_end) return;
  const int64_t z = min(static_cast<int64_t>(p.zero_end[b]), p.N_out);
  for (int64_t j = max(mv.s + mv.count, int64_t(0)) + first; j < z; j += step) dst[j] = 0.f;
}

// Into other tensors: a block takes kApartRows entries of a list, K and V. UNITS: 16-byte
// units of a row (0: any number).
constexpr int kApartRows = 64;
template <int UNITS>
__global__ void __launch_bounds__(kMoveThreads) mfa_compact_kernel(const __grid_constant__ CompactParams p) {
  __shared__ int64_t s_row[kApartRows];
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int g = blockIdx.y, b = blockIdx.z, units = UNITS > 0 ? UNITS : p.units;
  const Moves mv(p, g, b);
  const int base = blockIdx.x * kApartRows;
  float* w_out = p.w_out ? p.w_out + (static_cast<int64_t>(b) * p.Hkv + g) * p.N_out : nullptr;
  if (w_out) zero_tail(p, mv, w_out, b, blockIdx.x * kMoveThreads + threadIdx.x, static_cast<int64_t>(gridDim.x) * kMoveThreads);
  if (base >= mv.count) return;
  if (threadIdx.x < kApartRows) {
    const int t = base + threadIdx.x;
    const int64_t r = t < mv.count ? mv.source(p, t) : -1;
    s_row[threadIdx.x] = r;
    if (w_out && r >= 0) w_out[mv.s + t] = p.w[(static_cast<int64_t>(b) * p.Hkv + g) * p.N + r];
  }
  __syncthreads();
  const uint4* ks = p.k + b * p.ks[0] + g * p.ks[1];
  const uint4* vs = p.v + b * p.vs[0] + g * p.vs[1];
  uint4* ko = p.k_out + b * p.kos[0] + g * p.kos[1] + (mv.s + base) * p.kos[2];
  uint4* vo = p.v_out + b * p.vos[0] + g * p.vos[1] + (mv.s + base) * p.vos[2];
  constexpr int kBatch = 4;
  for (int i0 = threadIdx.x; i0 < kApartRows * units; i0 += kBatch * kMoveThreads) {
    uint4 x[kBatch], y[kBatch];
    int64_t r[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int e = i0 + i * kMoveThreads, t = e / units, u = e - t * units;
      r[i] = e < kApartRows * units ? s_row[t] : -1;
      if (r[i] >= 0) {
        x[i] = ks[r[i] * p.ks[2] + u];
        y[i] = vs[r[i] * p.vs[2] + u];
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int e = i0 + i * kMoveThreads, t = e / units, u = e - t * units;
      if (r[i] >= 0) {
        ko[t * p.kos[2] + u] = x[i];
        vo[t * p.vos[2] + u] = y[i];
      }
    }
  }
}

// In place. The destinations are the sources of earlier or the same entries
// only (idx[t] >= t), so a block that takes the entries in order, a chunk at a
// time, and loads a whole chunk before it stores any of it, reads every row
// before it is overwritten; the next chunk's rows lie behind all that this
// one writes, so they are loaded before, and the list one chunk earlier still. Blocks share
// nothing: each moves its own slice of the columns of one head's K or V, one more block the weights.
// Entries per thread and chunk (BATCH): 8 for long lists (64 lists of 8192 of 32768 rows of
// 128: 101 us, 5.4 TB/s; with 4, or slices of 8 or 16 units, 104 to 157 us), 2 where
// that takes the whole list in a chunk (6 rows of 64 heads: 3.8 us against 9.9, as more blocks fit an SM).
constexpr int kSlice = 4;   // 16-byte units of a row per block
constexpr int kShort = 2 * (kMoveThreads / kSlice);

// Moves a block's list: the thread's entries are first, first + step, ...; its rows' data are at[row * pitch].
template <int BATCH, typename T>
__device__ __forceinline__ void move_in_order(const CompactParams& p, const Moves& mv, int first, int step, T* at, int64_t pitch, bool mine,
                                              bool report) {
  const int count = mv.count, chunk = BATCH * step;
  int id[2][BATCH];
  T x[2][BATCH];
  unsigned have[2] = {0u, 0u};
  auto list = [&](int base, int (&v)[BATCH]) {
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int t = base + first + i * step;
      v[i] = t < count ? mv.idx[t] : 0;
    }
  };
  auto fetch = [&](int base, const int (&v)[BATCH], T (&y)[BATCH]) {
    unsigned moves = 0, bad = 0;
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int t = base + first + i * step;
      const int64_t r = mv.s + v[i], to = mv.s + t;
      const bool in = t < count, good = v[i] >= t && r >= 0 && r < p.N && to >= 0 && to < p.N_out;
      bad |= in && !good;
      moves |= (mine && in && good && v[i] != t ? 1u : 0u) << i;
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (moves >> i & 1) y[i] = at[(mv.s + v[i]) * pitch];
    if (bad && report) atomicOr(p.err, MFA_DEVERR_SEL);
    return moves;
  };
  auto put = [&](int base, const T (&y)[BATCH], unsigned moves) {
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (moves >> i & 1) at[(mv.s + base + first + i * step) * pitch] = y[i];
  };
  list(0, id[0]);
  list(chunk, id[1]);
  have[0] = fetch(0, id[0], x[0]);
  for (int base = 0; base < count; base += 2 * chunk) {
    __syncthreads();
    have[1] = fetch(base + chunk, id[1], x[1]);
    list(base + 2 * chunk, id[0]);
    put(base, x[0], have[0]);
    __syncthreads();
    have[0] = fetch(base + 2 * chunk, id[0], x[0]);
    list(base + 3 * chunk, id[1]);
    put(base + chunk, x[1], have[1]);
  }
}

template <int BATCH>
__global__ void __launch_bounds__(kMoveThreads) mfa_compact_in_place_kernel(const __grid_constant__ CompactParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int g = blockIdx.y, b = blockIdx.z;
  const int slices = (p.units + kSlice - 1) / kSlice;
  const Moves mv(p, g, b);
  if (blockIdx.x < 2 * slices) {
    const bool isv = blockIdx.x >= slices;
    const int slice = blockIdx.x - (isv ? slices : 0);
    const int u = slice * kSlice + threadIdx.x % kSlice;
    uint4* at = isv ? p.v_out + b * p.vs[0] + g * p.vs[1] + u : p.k_out + b * p.ks[0] + g * p.ks[1] + u;
    move_in_order<BATCH>(p, mv, static_cast<int>(threadIdx.x) / kSlice, kMoveThreads / kSlice, at, isv ? p.vs[2] : p.ks[2], u < p.units, blockIdx.x == 0);
  } else {
    float* at = p.w_out + (static_cast<int64_t>(b) * p.Hkv + g) * p.N;
    move_in_order<BATCH>(p, mv, static_cast<int>(threadIdx.x), kMoveThreads, at, int64_t(1), true, false);
    __syncthreads();
    zero_tail(p, mv, at, b, threadIdx.x, kMoveThreads);
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
// Whether a row of a and a row of b share bytes: a, b [B, H, N, D] of the same sizes with strides s and t,
// d the elements from a's first row to b's. They do where |d + sum_x (j_x t_x - i_x s_x)| < D for
// some 0 <= i_x, j_x < n_x. The steps are taken from the largest on, each as often as
// leaves a rest that the smaller ones can reach: once or twice in layouts that are
// permutations or slices of a dense one. (Others may take many; those beyond kTries count as sharing.)
struct Steps {
  int64_t step, lo, hi;  // taken lo to hi times
};
bool reaches(const Steps* at, int n, int64_t d, int64_t D, int* tries) {
  if (n == 0) return d > -D && d < D;
  int64_t lo = -D + 1 - d, hi = D - 1 - d;  // what the steps have to come to
  for (int x = 1; x < n; ++x) {
    lo -= at[x].hi * at[x].step;
    hi -= at[x].lo * at[x].step;
  }
  const int64_t s = at[0].step;
  const int64_t first = lo <= 0 ? -(-lo / s) : (lo + s - 1) / s, last = hi >= 0 ? hi / s : -((-hi + s - 1) / s);
  for (int64_t m = std::max(first, at[0].lo); m <= std::min(last, at[0].hi); ++m)
    if (--*tries < 0 || reaches(at + 1, n - 1, d + m * s, D, tries)) return true;
  return false;
}
bool share_row(const mfa_tensor* a, const mfa_tensor* b) {
  constexpr int kTries = 1 << 14;
  if (!overlap(tensor_range(a), tensor_range(b))) return false;
  const int64_t count[3] = {a->B, a->H, a->N};
  Steps at[6];
  int n = 0, tries = kTries;
  for (int x = 0; x < 3; ++x) {
    if (count[x] == 1) continue;
    const bool same = a->stride[x] == b->stride[x];
    at[n++] = {b->stride[x], same ? 1 - count[x] : 0, count[x] - 1};
    if (!same) at[n++] = {a->stride[x], 1 - count[x], 0};
  }
  std::sort(at, at + n, [](const Steps& x, const Steps& y) { return x.step > y.step; });
  const int64_t d = (reinterpret_cast<intptr_t>(b->data) - reinterpret_cast<intptr_t>(a->data)) / 2;  // (both on 16 bytes)
  return reaches(at, n, d, a->D, &tries);
}
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
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const int64_t keys = cdiv64(N, kSelWarps * kRun) * kSelWarps * kRun;  // with every warp's run full
  const dim3 grid(Hkv, B);
  bool ok;
  if (keys + budget <= kSelShared) {
    static std::atomic<uint64_t> attr_devs{0};
    if (!ensure_smem_attr(reinterpret_cast<const void*>(mfa_select_kernel<true, true>), kSelShared * 4, attr_devs)) return MFA_ERR_CUDA;
    ok = launch_after(mfa_select_kernel<true, true>, grid, kSelThreads, static_cast<size_t>(keys + budget) * 4, cs, p);
  } else if (keys <= kSelShared) {
    static std::atomic<uint64_t> attr_devs{0};
    if (!ensure_smem_attr(reinterpret_cast<const void*>(mfa_select_kernel<true, false>), kSelShared * 4, attr_devs)) return MFA_ERR_CUDA;
    ok = launch_after(mfa_select_kernel<true, false>, grid, kSelThreads, static_cast<size_t>(keys) * 4, cs, p);
  } else {
    ok = launch_after(mfa_select_kernel<false, false>, grid, kSelThreads, 0, cs, p);
  }
  return ok ? MFA_OK : MFA_ERR_CUDA;
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
  if (k->B > 65535 || k->H > 65535 || k->N >= (int64_t(1) << 30) || k_out->N >= (int64_t(1) << 30) || n_idx >= (1 << 30))
    return MFA_ERR_UNSUPPORTED;
  if (k->B == 0 || k->N == 0 || k_out->N == 0) return MFA_OK;
  if (!count || (!idx && n_idx > 0)) return MFA_ERR_INVALID_ARG;
  const bool in_place = same_tensor(k, k_out);
  if (in_place != same_tensor(v, v_out)) return MFA_ERR_INVALID_ARG;
  const Range rk = tensor_range(k), rv = tensor_range(v), ro = tensor_range(k_out), rp = tensor_range(v_out);
  if (in_place) {
    // (Interleaved caches, K and V of a token side by side, overlap as ranges but share no row.)
    if (share_row(k, v)) return MFA_ERR_INVALID_ARG;
  } else if (overlap(rk, ro) || overlap(rk, rp) || overlap(rv, ro) || overlap(rv, rp) || share_row(k_out, v_out)) {
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
  p.units = static_cast<int32_t>(k->D / 8); p.N = k->N; p.N_out = k_out->N;
  p.k = static_cast<const uint4*>(k->data); p.v = static_cast<const uint4*>(v->data);
  p.k_out = static_cast<uint4*>(k_out->data); p.v_out = static_cast<uint4*>(v_out->data);
  for (int a = 0; a < 3; ++a) {
    p.ks[a] = k->stride[a] / 8; p.vs[a] = v->stride[a] / 8;
    p.kos[a] = k_out->stride[a] / 8; p.vos[a] = v_out->stride[a] / 8;
  }
  p.w = weights; p.w_out = weights_out;
  p.start = start; p.idx = idx; p.count = count; p.zero_end = zero_end; p.err = dev_err;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (in_place) {
    const int slices = (p.units + kSlice - 1) / kSlice;
    const dim3 grid(2 * slices + (weights ? 1 : 0), p.Hkv, p.B);
    return launch_after(n_idx <= kShort ? mfa_compact_in_place_kernel<2> : mfa_compact_in_place_kernel<8>, grid, kMoveThreads, 0, cs, p)
               ? MFA_OK : MFA_ERR_CUDA;
  }
  const dim3 grid(static_cast<unsigned>(n_idx > 0 ? cdiv64(n_idx, kApartRows) : 1), p.Hkv, p.B);
  auto* kernel = p.units == 8 ? mfa_compact_kernel<8> : p.units == 16 ? mfa_compact_kernel<16>
               : p.units == 32 ? mfa_compact_kernel<32> : mfa_compact_kernel<0>;
  return launch_after(kernel, grid, kMoveThreads, 0, cs, p) ? MFA_OK : MFA_ERR_CUDA;
}

// mfa_tree_decode: attention of a tree of drafted tokens over a cache.
//
// out[b, h, t] = sum_j p_j v_j with p = softmax over the keys j the row sees of
// q . k_j / sqrt(D): every key before lens[b], and of the drafted ones behind
// it node t itself and its ancestors. The R = T * G rows of a key/value head
// (row t * G + h') read the same keys, so K and V are read once for up to 128
// rows; with more rows the CTAs of the row tiles walk the same keys side by
// side and share them in L2. Up to about 200 rows the work is bound by HBM.
//
// The products are transposed, S^T = K Q^T and O^T += V^T P^T, so that the 128
// rows of a tcgen05 MMA are 128 keys (or D columns) and its N is the number of
// query rows, 16 to 128: a decoded token pays for 16 rows, not 128, and a
// thread holds the scores of ONE key for all rows. The softmax then has no
// work along a thread's registers: the running maximum of a row is shared by
// the threads through shared memory and only checked (one comparison chain
// and one barrier vote per 128 keys); it moves when a score exceeds it by
// more than 8 (2^8 fits every type here), and the sums stay per thread until
// the end. P^T goes to shared memory as bf16 (the tensor core's input type; half a step
// of each weight), where it lies as the MMA's B operand wants it.
//
// The tiles (128 keys) of all (batch, head) pairs are laid end to end and cut
// into equal ranges, one per CTA, from the lengths on the device: the grid
// does not depend on them. A pair met by one CTA is written directly; of a
// pair cut between CTAs each writes an unnormalised part (m, l, o), and a
// dependent launch merges them in a fixed order.
#include <cfloat>
#include <cmath>
#include <cuda_bf16.h>

#include "cache.cuh"
#include "mfa_device.cuh"

namespace mfa {
namespace {

constexpr int kKeys = 128;           // keys per tile
constexpr int kChunk = kKeys * 128;  // bytes of 64 columns of a tile, 128-byte swizzled rows
constexpr int kMaxRows = 128;        // query rows per row tile
constexpr float kLazy = 8.0f;        // a row's maximum moves when a score exceeds it by this (in powers of two)

struct TreeParams {
  int32_t B, Hq, Hkv, G, T, N, R;  // R = T * G rows per key/value head
  int32_t rtiles, groups;          // row tiles; CTAs per row tile
  float scale_log2;
  const __nv_bfloat16* q;
  int64_t qs[3], os[3];
  const int32_t *lens, *parents;
  __nv_bfloat16* out;
  float *lse, *o_part, *ml_part;  // parts: [rtiles * groups][2][NR][D] and [..][NR][2] (m, l)
  uint32_t* err;
};

// Tiles of a (batch, head) pair for row tile rt: up to the last node its rows can see.
template <int NR>
__device__ __forceinline__ int tiles_of(const TreeParams& p, int len, int rt) {
  const int t_hi = min((rt * NR + NR - 1) / p.G, p.T - 1);
  return (min(len + t_hi + 1, p.N) + kKeys - 1) / kKeys;
}

// ---------------------------------------------------------------------------
// Where a CTA's range begins. All of the block's threads call it: every thread
// sums the tiles of a run of batches, a scan gives the total and finds the
// batch that holds tile index `at(total)`.
// ---------------------------------------------------------------------------
struct Start {
  int64_t total, begin, before;  // tiles of the row tile's line; first of this CTA; first of batch b
  int32_t b;
};

template <int NR, int THREADS, typename At>
__device__ __forceinline__ void find_start(const TreeParams& p, int rt, Start* s, int64_t* scan, At at) {
  const int per = (p.B + THREADS - 1) / THREADS;
  const int b0 = min(static_cast<int>(threadIdx.x) * per, p.B), b1 = min(b0 + per, p.B);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += tiles_of<NR>(p, cache_len(p.lens, b, p.N), rt);
  int64_t sum = mine;
#pragma unroll
  for (int w = 1; w < 32; w <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, sum, w);
    if (lane >= w) sum += o;
  }
  if (lane == 31) scan[warp] = sum;
  __syncthreads();
  int64_t base = 0, total = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) base += scan[w];
    total += scan[w];
  }
  total *= p.Hkv;
  const int64_t begin = at(total);
  int64_t first = (base + sum - mine) * p.Hkv;  // of batch b0
  if (threadIdx.x == 0) {
    s->total = total;
    s->begin = begin;
    s->b = -1;
  }
  __syncthreads();
  if (begin >= first && begin < first + mine * p.Hkv) {
    for (int b = b0; b < b1; ++b) {
      const int64_t n = static_cast<int64_t>(tiles_of<NR>(p, cache_len(p.lens, b, p.N), rt)) * p.Hkv;
      if (begin < first + n) {
        s->before = first;
        s->b = b;
        break;
      }
      first += n;
    }
  }
  __syncthreads();
}

__device__ __forceinline__ int64_t tiles_per_cta(int64_t total, int groups) { return (total + groups - 1) / groups; }

// The (batch, head) pairs of a CTA's range, one after the other.
template <int NR>
struct Walk {
  int b, g, t0, t1, len, nt;
  int64_t left;  // tiles of the range not yet given out
  __device__ __forceinline__ Walk(const TreeParams& p, int rt, const Start& s) {
    const int64_t per = tiles_per_cta(s.total, p.groups);
    left = min(per, s.total - s.begin);
    b = s.b;
    len = cache_len(p.lens, b, p.N);
    nt = tiles_of<NR>(p, len, rt);
    const int64_t in = s.begin - s.before;
    g = static_cast<int>(in / nt);
    t0 = static_cast<int>(in % nt);
    t1 = static_cast<int>(min(static_cast<int64_t>(nt), t0 + left));
    left -= t1 - t0;
  }
  // The next pair; false at the range's end.
  __device__ __forceinline__ bool next(const TreeParams& p, int rt) {
    if (left <= 0) return false;
    if (++g == p.Hkv) {
      g = 0;
      ++b;
      len = cache_len(p.lens, b, p.N);
      nt = tiles_of<NR>(p, len, rt);
    }
    t0 = 0;
    t1 = static_cast<int>(min(static_cast<int64_t>(nt), left));
    left -= t1;
    return true;
  }
};

// ---------------------------------------------------------------------------
// Layout. K and V come in units of 128 keys x 128 columns (64 for D = 64)
// through one ring, a tile's K units before its V units. P's buffer is also
// the scratch of everything rare (each softmax group its own 16 KB of it).
// ---------------------------------------------------------------------------
template <int D, int NR>
struct Cfg {
  static constexpr int kSoftWarps = NR == 128 ? 8 : 4;  // a group of 4 warps takes 64 rows
  static constexpr int kGroups = kSoftWarps / 4;
  static constexpr int kCols = NR / kGroups;            // rows (registers) per thread
  static constexpr int kThreads = (kSoftWarps + 2) * 32;
  static constexpr int kUnits = D == 256 ? 2 : 1;       // ring units of a K (or V) tile
  static constexpr int kUnit = (D == 64 ? 1 : 2) * kChunk;
  static constexpr int kPBytes = kGroups * kChunk;
  static constexpr int kPBufs = NR == 128 && D > 64 ? 1 : 2;
  static constexpr int kRing = D == 64 ? 8 : (D == 256 && NR == 128 ? 4 : 5);
  static constexpr int kQ = 0;                          // NR rows x 128 B per 64 columns
  static constexpr int kQBytes = NR * D * 2;
  static constexpr int kRing0 = (kQBytes + 1023) / 1024 * 1024;
  static constexpr int kP = kRing0 + kRing * kUnit;     // behind the ring: D = 64 reads one chunk past its last unit
  static constexpr int kMisc = kP + kPBufs * kPBytes;
  static constexpr int kMiscBytes = 2048;
  static constexpr int kBytes = kMisc + kMiscBytes + 1024;  // + slack for 1024-byte alignment
  static constexpr int kO = 2 * NR;                     // TMEM columns: S0 [0, NR) S1 [NR, 2 NR) O [2 NR, (2 + kUnits) NR)
  static constexpr int kTmem = 4 * NR;
  static_assert(kBytes <= 232448, "shared memory");
  static_assert(kTmem <= 512, "TMEM columns");
};

// D[tmem] = A B^T with both operands in shared memory; A and B K-major or both MN-major.
__host__ __device__ constexpr uint32_t idesc_tree(int N, bool mn_major) {
  return idesc_bf16_f32(128, N, mn_major) | (mn_major ? 1u << 15 : 0u);
}

__device__ __forceinline__ bool vote_or(uint32_t id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r) : "r"(x ? 1u : 0u), "r"(id) : "memory");
  return r != 0;
}
__device__ __forceinline__ float warp_max(float x) {  // NaN is ignored unless all are
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

template <int C>
__device__ __forceinline__ void tmem_ld_cols(uint32_t addr, float (&x)[C]) {
  if constexpr (C == 16) {
    uint32_t r[16];
    tmem_ld_32x32b_x16(addr, r);
    tmem_ld_wait();
#pragma unroll
    for (int c = 0; c < 16; ++c) x[c] = __uint_as_float(r[c]);
  } else {
    uint32_t r[C / 32][32];
#pragma unroll
    for (int k = 0; k < C / 32; ++k) tmem_ld_32x32b_x32(addr + k * 32, r[k]);
    tmem_ld_wait();
#pragma unroll
    for (int c = 0; c < C; ++c) x[c] = __uint_as_float(r[c >> 5][c & 31]);
  }
}

// Sums v[c] over the warp's lanes: in five halvings lane l ends with the sums
// of the C / 32 (or, repeated, one) values number first + ...; returns first.
template <int C>
__device__ __forceinline__ int warp_sum_spread(float (&v)[C], int lane) {
  int first = 0;
  int n = C;
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool up = lane & w;
#pragma unroll
      for (int c = 0; c < C / 2; ++c) {
        if (c < n) {
          const float give = up ? v[c] : v[c + n], keep = up ? v[c + n] : v[c];
          v[c] = keep + __shfl_xor_sync(0xffffffffu, give, w);
        }
      }
      first += up ? n : 0;
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], w);
    }
  }
  return first;
}

template <int D, int NR>
__global__ void __launch_bounds__(Cfg<D, NR>::kThreads, 1)
    mfa_tree_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ TreeParams p) {
  using C = Cfg<D, NR>;
  constexpr int U = C::kUnits, RING = C::kRing, PB = C::kPBufs, W = C::kCols;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rt = blockIdx.x % p.rtiles, cta = blockIdx.x / p.rtiles;

  float* sNegM = reinterpret_cast<float*>(smem + C::kMisc);  // [NR] minus the row's maximum; 0 while it has none
  float* sDelta = sNegM + NR;                                // [NR] how far it moved; at the end 1 / l
  float* sAlpha = sDelta + NR;                               // [NR] 2^-delta
  uint8_t* sSet = reinterpret_cast<uint8_t*>(sAlpha + NR);   // [NR] the row has a maximum
  uint8_t* sPoison = sSet + NR;                              // [NR] the row sees a value that is not finite
  uint64_t* bars = reinterpret_cast<uint64_t*>(sPoison + NR);
  uint64_t* full = bars;               // [RING]
  uint64_t* empty = full + RING;       // [RING]
  uint64_t* q_full = empty + RING;     // Q of the next pair is in shared memory
  uint64_t* s_full = q_full + 1;       // [2]
  uint64_t* s_empty = s_full + 2;      // [2] read into registers
  uint64_t* p_full = s_empty + 2;      // [PB]
  uint64_t* p_empty = p_full + 2;      // [PB] P.V done
  uint64_t* drain = p_empty + 2;
  Start* sStart = reinterpret_cast<Start*>(drain + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(sStart + 1);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(const_cast<int*>(s_abort) + 1);
  static_assert(NR * 14 + (2 * RING + 10) * 8 + sizeof(Start) + 8 <= C::kMiscBytes, "misc");

  // The merging kernel may be scheduled now: it waits for this grid to end.
  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x == 0) {
    for (int i = 0; i < RING; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], C::kSoftWarps * 32);
      mbar_init(&p_full[i], C::kSoftWarps * 32);
      mbar_init(&p_empty[i], 1);
    }
    mbar_init(q_full, C::kSoftWarps * 32);
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_mbarrier_init();
  }
  find_start<NR, C::kThreads>(p, rt, sStart, reinterpret_cast<int64_t*>(smem + C::kP),
                              [&](int64_t total) { return cta * tiles_per_cta(total, p.groups); });
  const Start start = *sStart;
  if (start.begin >= start.total) return;  // more CTAs than tiles
  if (warp == C::kSoftWarps) {
    tmem_alloc(s_tmem, C::kTmem);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const int total = static_cast<int>(min(tiles_per_cta(start.total, p.groups), start.total - start.begin));

  if (warp == C::kSoftWarps + 1) {
    // =================== TMA producer ===================
    if (lane == 0) {
      Walk<NR> w(p, rt, start);
      uint32_t idx = 0;  // units issued
      bool ok = true;
      do {
        for (int t = w.t0; t < w.t1 && ok; ++t) {
#pragma unroll
          for (int u = 0; u < 2 * U; ++u) {
            const uint32_t slot = idx % RING;
            if (idx >= RING && !(ok = mbar_wait(&empty[slot], (idx / RING - 1) & 1, s_abort))) break;
            mbar_arrive_expect_tx(&full[slot], C::kUnit);
            uint8_t* dst = smem + C::kRing0 + slot * C::kUnit;
            const CUtensorMap* map = u < U ? &tm_k : &tm_v;
#pragma unroll
            for (int c = 0; c < C::kUnit / kChunk; ++c)
              tma_load_4d(dst + c * kChunk, map, &full[slot], (u % U) * 128 + c * 64, t * kKeys, w.g, w.b);
            ++idx;
          }
        }
      } while (ok && w.next(p, rt));
      if (*s_abort) {
        // Loads in flight land before the CTA exits.
        volatile int no_abort = 0;
        for (uint32_t j = idx > RING ? idx - RING : 0; j < idx; ++j) mbar_wait(&full[j % RING], (j / RING) & 1, &no_abort);
      }
    }
  } else if (warp == C::kSoftWarps) {
    // =================== MMA issuer ===================
    constexpr uint32_t idesc_s = idesc_tree(NR, false), idesc_o = idesc_tree(NR, true);
    const uint32_t ring = smem_u32(smem + C::kRing0), q_addr = smem_u32(smem + C::kQ), p_addr = smem_u32(smem + C::kP);
    Walk<NR> ws(p, rt, start), wp(p, rt, start);
    int ts = ws.t0, tp = wp.t0;           // tiles of the next S and the next P.V
    int ns = 0, np = 0, seg = 0;          // S and P.V issued; pairs begun
    bool fresh_s = true, fresh_p = true;  // the next one is its pair's first
    bool ok = true;
    uint64_t t_idle = 0;
    auto have = [&](uint32_t first) {  // the U units from ring index `first` on have landed
      bool x = true;
#pragma unroll
      for (int u = 0; u < U; ++u) x &= mbar_test_wait(&full[(first + u) % RING], ((first + u) / RING) & 1);
      return __all_sync(0xffffffffu, x) != 0;
    };
    // Whichever is ready first goes out: the next S, or the oldest pending P.V.
    while (ok && np < total) {
      bool did = false;
      if (ns < total && ns <= np + 1) {
        const uint32_t first = static_cast<uint32_t>(ns) * 2 * U;
        if ((!fresh_s || __all_sync(0xffffffffu, mbar_test_wait(q_full, seg & 1))) &&
            (ns < 2 || __all_sync(0xffffffffu, mbar_test_wait(&s_empty[ns & 1], ((ns >> 1) - 1) & 1))) && have(first)) {
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t slot = (first + (kk >> 3)) % RING;
            const uint32_t ka = ring + slot * C::kUnit + ((kk >> 2) & (C::kUnit / kChunk - 1)) * kChunk + (kk & 3) * 32;
            const uint32_t qb = q_addr + (kk >> 2) * (NR * 128) + (kk & 3) * 32;
            umma_ss(tmem + (ns & 1) * NR, sdesc_sw128_lo(ka, 16), sdesc_sw128_lo(qb, 16), idesc_s, kk > 0 ? 1u : 0u);
          }
          umma_commit(&s_full[ns & 1]);
#pragma unroll
          for (int u = 0; u < U; ++u) umma_commit(&empty[(first + u) % RING]);
          ++ns;
          did = true;
          fresh_s = false;
          if (++ts == ws.t1 && ws.next(p, rt)) {
            ts = ws.t0;
            fresh_s = true;
            ++seg;
          }
        }
      }
      if (!did && np < ns) {
        const uint32_t first = static_cast<uint32_t>(np) * 2 * U + U;
        if (__all_sync(0xffffffffu, mbar_test_wait(&p_full[np % PB], (np / PB) & 1)) && have(first)) {
          tc_fence_after();
          const uint32_t pb = sdesc_sw128_lo(p_addr + (np % PB) * C::kPBytes, kChunk);
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const uint32_t va = sdesc_sw128_lo(ring + ((first + u) % RING) * C::kUnit, kChunk);
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              umma_ss(tmem + C::kO + u * NR, va + kk * (16 * 128 / 16), pb + kk * (16 * 128 / 16), idesc_o,
                      (!fresh_p || kk > 0) ? 1u : 0u);
          }
          umma_commit(&p_empty[np % PB]);
#pragma unroll
          for (int u = 0; u < U; ++u) umma_commit(&empty[(first + u) % RING]);
          ++np;
          did = true;
          fresh_p = false;
          if (++tp == wp.t1 && wp.next(p, rt)) {
            tp = wp.t0;
            fresh_p = true;
          }
        }
      }
      if (did) {
        t_idle = 0;
      } else {
        // Bounded like every other wait.
        if (*s_abort) ok = false;
        const uint64_t now = global_timer_ns();
        if (t_idle == 0) t_idle = now;
        else if (now - t_idle > kWaitTimeoutNs) ok = false;
        ok = __all_sync(0xffffffffu, ok);
      }
    }
    if (!ok) *s_abort = 1;
    umma_commit(drain);
    volatile int no_abort = 0;
    mbar_wait(drain, 0, &no_abort);
  } else {
    // =================== softmax and epilogue: a thread per key ===================
    // A failed wait raises *s_abort and the thread runs on (every later wait
    // then fails at once): the barriers below need all of the group's threads.
    const int grp = warp >> 2, quad = warp & 3;
    const int tid = quad * 32 + lane;           // key of the tile; column of D
    const uint32_t bar = 1 + grp;               // the group's named barrier
    const int col0 = grp * W;                   // its first row of the tile
    const uint32_t tm = tmem + (static_cast<uint32_t>(quad * 32) << 16) + col0;
    const int row0 = rt * NR + col0;            // its first row of the pair
    const int rows = min(W, p.R - row0);        // real ones (may be <= 0)
    const float* negM = sNegM + col0;
    float* delta = sDelta + col0;
    float* alpha = sAlpha + col0;
    Walk<NR> w(p, rt, start);
    int n = 0;
    do {
      // ---- Q of the pair, zeros for rows that are none (every S of the previous pair is done) ----
      const int32_t* par = p.parents ? p.parents + static_cast<int64_t>(w.b) * p.T : nullptr;
      for (int i = threadIdx.x; i < NR * (D / 8); i += C::kSoftWarps * 32) {
        const int r = i / (D / 8), u = i % (D / 8), row = rt * NR + r;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (row < p.R) {
          const int t = row / p.G, h = w.g * p.G + row % p.G;
          if (!par || __ldg(par + t) != -2)
            x = __ldg(reinterpret_cast<const uint4*>(p.q + w.b * p.qs[0] + h * p.qs[1] + t * p.qs[2]) + u);
        }
        *reinterpret_cast<uint4*>(smem + C::kQ + (u >> 3) * (NR * 128) + r * 128 + (((u & 7) ^ (r & 7)) << 4)) = x;
      }
      if (tid < W) {
        sNegM[col0 + tid] = 0.f;
        sSet[col0 + tid] = 0;
        sPoison[col0 + tid] = 0;
      }
      if (rt == 0 && w.g == 0 && w.t0 == 0) {
        for (int t = threadIdx.x; t < (par ? p.T : 1); t += C::kSoftWarps * 32) {
          const uint32_t e = draft_errors(p.lens, p.parents, w.b, t, p.T, p.N);
          if (e) atomicOr(p.err, e);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(q_full);
      named_barrier(bar, 128);
      uint64_t l[W / 2];
#pragma unroll
      for (int c = 0; c < W / 2; ++c) l[c] = 0ull;

      for (int t = w.t0; t < w.t1; ++t, ++n) {
        const int base = t * kKeys;
        float x[W];
        mbar_wait(&s_full[n & 1], (n >> 1) & 1, s_abort);
        tc_fence_after();
        tmem_ld_cols<W>(tm + (n & 1) * NR, x);
        tc_fence_before();
        mbar_arrive(&s_empty[n & 1]);
        uint8_t* pbuf = smem + C::kP + (n % PB) * C::kPBytes + grp * kChunk;  // the group's 64 columns of P
        const bool draft = base + kKeys > w.len;
        if (draft) {
          // ---- a tile with drafted keys, or the last: who sees what ----
          mbar_wait(&p_empty[n % PB], ((n / PB) - 1) & 1, s_abort);  // pbuf is free (passes while it was never used)
          const int j = base + tid, node = j - w.len;
          const bool held = j < min(w.len + p.T, p.N);
          int* sPar = reinterpret_cast<int*>(pbuf);
          uint32_t* sSeen = reinterpret_cast<uint32_t*>(pbuf + MFA_TREE_MAX_NODES * 4);  // [W][8]: the nodes a row sees
          if (par) {
            for (int i = tid; i < p.T; i += 128) sPar[i] = __ldg(par + i);
            named_barrier(bar, 128);
            if (tid < W) {
              uint32_t bits[MFA_TREE_MAX_NODES / 32] = {};
              const int tt = tid < rows ? (row0 + tid) / p.G : 0;
              if (tid < rows && sPar[tt] != -2)
                for (int a = tt; a >= 0; a = tree_up(sPar, a)) {
#pragma unroll
                  for (int k = 0; k < MFA_TREE_MAX_NODES / 32; ++k) bits[k] |= (a >> 5) == k ? 1u << (a & 31) : 0u;
                }
#pragma unroll
              for (int k = 0; k < MFA_TREE_MAX_NODES / 32; ++k) sSeen[tid * (MFA_TREE_MAX_NODES / 32) + k] = bits[k];
            }
            named_barrier(bar, 128);
          }
          // V of a key that is not before the sequence's end must be finite,
          // seen or not: 0 * inf would reach every row.
          // (A test of a ring slot's phase needs its last occupant's to be over:
          // it belongs to the tile before at the latest, whose P.V is awaited.)
          if (n > 0) mbar_wait(&p_empty[(n - 1) % PB], ((n - 1) / PB) & 1, s_abort);
          bool finite = true;
          if (j >= w.len) {
#pragma unroll 1
            for (int u = 0; u < D / 8; ++u) {
              const uint32_t unit = static_cast<uint32_t>(n) * 2 * U + U + (u >> 4);
              if ((u & 15) == 0) mbar_wait(&full[unit % RING], (unit / RING) & 1, s_abort);
              const uint4 y = *reinterpret_cast<const uint4*>(smem + C::kRing0 + (unit % RING) * C::kUnit + ((u >> 3) & 1) * kChunk +
                                                              tid * 128 + (((u & 7) ^ (tid & 7)) << 4));
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t v = k == 0 ? y.x : k == 1 ? y.y : k == 2 ? y.z : y.w;
                finite &= (v & 0x7f80u) != 0x7f80u && (v & 0x7f800000u) != 0x7f800000u;
              }
            }
          }
          int tt = row0 / p.G, hh = row0 % p.G;
#pragma unroll
          for (int c = 0; c < W; ++c) {
            if (j >= w.len) {
              bool see = held && c < rows;
              if (see) see = par ? (sSeen[c * (MFA_TREE_MAX_NODES / 32) + (node >> 5)] >> (node & 31)) & 1 : node <= tt;
              if (!see) x[c] = -INFINITY;
              else if (!finite) sPoison[col0 + c] = 1;
            }
            if (++hh == p.G) {
              hh = 0;
              ++tt;
            }
          }
          named_barrier(3, C::kSoftWarps * 32);  // both groups have looked
          if (j >= w.len && !(held && finite) && grp == 0) {
#pragma unroll 1
            for (int u = 0; u < D / 8; ++u) {
              const uint32_t unit = static_cast<uint32_t>(n) * 2 * U + U + (u >> 4);
              *reinterpret_cast<uint4*>(smem + C::kRing0 + (unit % RING) * C::kUnit + ((u >> 3) & 1) * kChunk + tid * 128 +
                                        (((u & 7) ^ (tid & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
            }
          }
        }
        // ---- scores in powers of two, relative to the rows' maxima ----
        const uint64_t sc2 = f2_pack(p.scale_log2, p.scale_log2);
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < W; c += 4) {
          const ulonglong2 nm = *reinterpret_cast<const ulonglong2*>(negM + c);
          f2_unpack(f2_fma(f2_pack(x[c], x[c + 1]), sc2, nm.x), x[c], x[c + 1]);
          f2_unpack(f2_fma(f2_pack(x[c + 2], x[c + 3]), sc2, nm.y), x[c + 2], x[c + 3]);
          mx[0] = fmax3(mx[0], x[c], x[c + 1]);
          mx[1] = fmax3(mx[1], x[c + 2], x[c + 3]);
        }
        const bool first = t == w.t0;
        if (vote_or(bar, fmaxf(mx[0], mx[1]) > kLazy) || first || draft) {
          // ---- rare: new maxima ----
          if (!draft) mbar_wait(&p_empty[n % PB], ((n / PB) - 1) & 1, s_abort);  // (passes while the buffer was never used)
          float* sMax = reinterpret_cast<float*>(pbuf);  // [4][W]
#pragma unroll
          for (int c = 0; c < W; ++c) {
            const float m = warp_max(x[c]);
            if (lane == (c & 31)) sMax[quad * W + c] = m;
          }
          named_barrier(bar, 128);
          bool moved = false;
          if (tid < W) {
            const float m = fmaxf(fmaxf(sMax[tid], sMax[W + tid]), fmaxf(sMax[2 * W + tid], sMax[3 * W + tid]));
            const bool set = sSet[col0 + tid] != 0;
            float d = 0.f;
            if (m > (set ? kLazy : -INFINITY)) {
              const float nm = sNegM[col0 + tid] - m;
              d = sNegM[col0 + tid] - nm;
              sNegM[col0 + tid] = nm;
              sSet[col0 + tid] = 1;
            }
            delta[tid] = d;
            alpha[tid] = set ? ex2_approx(-d) : 1.f;  // a row without a maximum has no sums yet
            moved = set && d != 0.f;
          }
          moved = vote_or(bar, moved);
#pragma unroll
          for (int c = 0; c < W; c += 2) {
            x[c] -= delta[c];
            x[c + 1] -= delta[c + 1];
          }
          if (moved) {
#pragma unroll
            for (int c = 0; c < W / 2; ++c) {
              float a, b;
              f2_unpack(l[c], a, b);
              l[c] = f2_pack(a * alpha[2 * c], b * alpha[2 * c + 1]);
            }
            // O holds every P.V of the pair before this tile's once the last is done.
            mbar_wait(&p_empty[(n - 1) % PB], ((n - 1) / PB) & 1, s_abort);
            tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < U * (W / 16); ++k) {
              const int c = (k % (W / 16)) * 16;
              const uint32_t at = tm + C::kO + (k / (W / 16)) * NR + c;
              uint32_t o[16];
              tmem_ld_32x32b_x16(at, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha[c + i]);
              tmem_st_32x32b_x16(at, o);
            }
            tmem_st_wait();
            tc_fence_before();
          }
        }
        // ---- weights: 2^x, their sums, and P in bf16 ----
        uint32_t pk[W / 2];
#pragma unroll
        for (int c = 0; c < W / 2; ++c) {
          const float e0 = ex2_approx(x[2 * c]), e1 = ex2_approx(x[2 * c + 1]);
          l[c] = f2_add(l[c], f2_pack(e0, e1));
          pk[c] = pack_bf16x2(e0, e1);
        }
        if (n >= PB) mbar_wait(&p_empty[n % PB], ((n / PB) - 1) & 1, s_abort);
#pragma unroll
        for (int u = 0; u < W / 8; ++u)
          *reinterpret_cast<uint4*>(pbuf + tid * 128 + ((u ^ (tid & 7)) << 4)) =
              make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
        fence_proxy_async_smem();
        mbar_arrive(&p_full[n % PB]);
      }

      // ---- epilogue of the pair: its output, or this CTA's part of it ----
      mbar_wait(&p_empty[(n - 1) % PB], ((n - 1) / PB) & 1, s_abort);
      tc_fence_after();
      const bool whole = w.t0 == 0 && w.t1 == w.nt;
      const int64_t part = (static_cast<int64_t>(blockIdx.x) * 2 + (w.t0 > 0 ? 0 : 1)) * NR + col0;
      float* sL = reinterpret_cast<float*>(smem + C::kP + grp * kChunk);  // [4][W]
      {
        float v[W];
#pragma unroll
        for (int c = 0; c < W / 2; ++c) f2_unpack(l[c], v[2 * c], v[2 * c + 1]);
        const int f = warp_sum_spread<W>(v, lane);
        if (W == 64) {
          sL[quad * W + f] = v[0];
          sL[quad * W + f + 1] = v[1];
        } else {
          sL[quad * W + f] = v[0];  // (W = 16: two lanes write the same value)
        }
      }
      named_barrier(bar, 128);
      if (tid < rows && tid < W) {
        const int tt = (row0 + tid) / p.G, h = w.g * p.G + (row0 + tid) % p.G;
        const bool dead = par && __ldg(par + tt) == -2;
        const float sum = dead ? 0.f : (sL[tid] + sL[W + tid]) + (sL[2 * W + tid] + sL[3 * W + tid]);
        const float m = -sNegM[col0 + tid];
        // What the row's outputs are multiplied by; -1: it has none.
        delta[tid] = sum == 0.f ? -1.f : (sPoison[col0 + tid] ? NAN : (whole ? 1.f / sum : 1.f));
        if (whole) {
          p.lse[(static_cast<int64_t>(w.b) * p.Hq + h) * p.T + tt] =
              sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.69314718055994530942f;
        } else {
          p.ml_part[(part + tid) * 2] = sum == 0.f ? -FLT_MAX : m;
          p.ml_part[(part + tid) * 2 + 1] = sum;
        }
      }
      named_barrier(bar, 128);
#pragma unroll 1
      for (int u = 0; u < U; ++u) {
        int tt = row0 / p.G, hh = row0 % p.G;
        const int d = u * 128 + tid;
#pragma unroll 1
        for (int c = 0; c < rows && c < W; c += 16) {
          uint32_t o[16];
          tmem_ld_32x32b_x16(tm + C::kO + u * NR + c, o);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (c + i < rows && d < D) {
              const float f = delta[c + i];
              const float y = f == -1.f ? 0.f : __uint_as_float(o[i]) * f;
              if (whole)
                p.out[w.b * p.os[0] + static_cast<int64_t>(w.g * p.G + hh) * p.os[1] + tt * p.os[2] + d] = __float2bfloat16_rn(y);
              else
                p.o_part[(part + c + i) * D + d] = y;
            }
            if (++hh == p.G) {
              hh = 0;
              ++tt;
            }
          }
        }
      }
      tc_fence_before();
      named_barrier(bar, 128);  // delta and the scratch are read before the next pair writes them
    } while (w.next(p, rt));
    if (*s_abort && threadIdx.x == 0) atomicOr(p.err, MFA_DEVERR_TIMEOUT);
  }
  __syncthreads();
  if (warp == C::kSoftWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// ---------------------------------------------------------------------------
// Merges the parts of every pair that was cut: with M = max m_s, out = sum o_s
// 2^(m_s - M) / sum l_s 2^(m_s - M). A part without a visible key has
// m = -FLT_MAX, l = 0, o = 0 (never -inf - -inf); all such: out = 0, lse = -inf.
// A block takes `rpb` rows of a pair, 8 (few parts: a warp-sized group of
// threads per row and its columns) or 1 (the groups split the parts).
// ---------------------------------------------------------------------------
constexpr int kMergeThreads = 256;

template <int D, int NR>
__global__ void __launch_bounds__(kMergeThreads) mfa_tree_merge(const __grid_constant__ TreeParams p, int rpb) {
  constexpr int L = D / 4, S = kMergeThreads / L;  // threads per row, groups
  __shared__ Start start;
  __shared__ int64_t scan[kMergeThreads / 32];
  __shared__ float4 so[S][L];
  __shared__ float sl[S];
  const int rt = blockIdx.y % p.rtiles, r0 = (blockIdx.y / p.rtiles) * rpb;  // rows of the row tile
  const int b = blockIdx.x / p.Hkv, g = blockIdx.x % p.Hkv;
  const int rows = min(NR, p.R - rt * NR);
  if (r0 >= rows) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // The pair's first tile on the row tile's line.
  int64_t before = 0;
  {
    int64_t mine = 0, all = 0;
    for (int x = threadIdx.x; x < p.B; x += kMergeThreads) {
      const int n = tiles_of<NR>(p, cache_len(p.lens, x, p.N), rt);
      all += n;
      if (x < b) mine += n;
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) {
      mine += __shfl_xor_sync(0xffffffffu, mine, w);
      all += __shfl_xor_sync(0xffffffffu, all, w);
    }
    if ((threadIdx.x & 31) == 0) {
      scan[threadIdx.x >> 5] = mine;
      reinterpret_cast<int64_t*>(so)[threadIdx.x >> 5] = all;
    }
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < kMergeThreads / 32; ++w) {
      before += scan[w];
      total += reinterpret_cast<int64_t*>(so)[w];
    }
    __syncthreads();
    if (threadIdx.x == 0) start.total = total * p.Hkv;
    __syncthreads();
  }
  const int nt = tiles_of<NR>(p, cache_len(p.lens, b, p.N), rt);
  const int64_t base = before * p.Hkv + static_cast<int64_t>(g) * nt;
  const int64_t per = tiles_per_cta(start.total, p.groups);
  const int64_t c0 = base / per, c1 = (base + nt - 1) / per;
  if (c0 == c1) return;  // written by its only CTA
  const int ns = static_cast<int>(c1 - c0 + 1);
  // Row r's part s.
  auto at = [&](int s, int r) {
    const int64_t c = c0 + s;
    return ((c * p.rtiles + rt) * 2 + (c * per > base ? 0 : 1)) * NR + r;
  };
  const int grp = threadIdx.x / L, d = (threadIdx.x % L) * 4;
  auto write = [&](int r, float4 o, float l, float M) {
    const int row = rt * NR + r, t = row / p.G, h = g * p.G + row % p.G;
    const bool has = l != 0.f;
    const float inv = has ? 1.f / l : 0.f;
    uint2 w = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (!has) w = make_uint2(0u, 0u);
    *reinterpret_cast<uint2*>(p.out + b * p.os[0] + h * p.os[1] + t * p.os[2] + d) = w;
    if (d == 0)
      p.lse[(static_cast<int64_t>(b) * p.Hq + h) * p.T + t] = has ? (M + log2f(l)) * 0.69314718055994530942f : -INFINITY;
  };
  if (rpb > 1) {
    for (int r = r0 + grp; r < min(r0 + rpb, rows); r += S) {
      float M = -FLT_MAX, l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int s = 0; s < ns; ++s) M = fmaxf(M, p.ml_part[at(s, r) * 2]);
#pragma unroll 4
      for (int s = 0; s < ns; ++s) {
        const int64_t x = at(s, r);
        const float2 ml = *reinterpret_cast<const float2*>(p.ml_part + x * 2);
        const float4 y = *reinterpret_cast<const float4*>(p.o_part + x * D + d);
        const float f = ex2_approx(ml.x - M);
        l = fmaf(f, ml.y, l);
        o.x = fmaf(f, y.x, o.x); o.y = fmaf(f, y.y, o.y); o.z = fmaf(f, y.z, o.z); o.w = fmaf(f, y.w, o.w);
      }
      write(r, o, l, M);
    }
    return;
  }
  float M = -FLT_MAX, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = 0; s < ns; ++s) M = fmaxf(M, p.ml_part[at(s, r0) * 2]);
#pragma unroll 4
  for (int s = grp; s < ns; s += S) {
    const int64_t x = at(s, r0);
    const float2 ml = *reinterpret_cast<const float2*>(p.ml_part + x * 2);
    const float4 y = *reinterpret_cast<const float4*>(p.o_part + x * D + d);
    const float f = ex2_approx(ml.x - M);
    l = fmaf(f, ml.y, l);
    o.x = fmaf(f, y.x, o.x); o.y = fmaf(f, y.y, o.y); o.z = fmaf(f, y.z, o.z); o.w = fmaf(f, y.w, o.w);
  }
  so[grp][d / 4] = o;
  if (d == 0) sl[grp] = l;
  __syncthreads();
  if (grp == 0) {
#pragma unroll
    for (int s = 1; s < S; ++s) {
      const float4 y = so[s][d / 4];
      o.x += y.x; o.y += y.y; o.z += y.z; o.w += y.w;
      l += sl[s];
    }
    write(r0, o, l, M);
  }
}

// ---- host ----

struct TreePlan {
  int nr, rtiles, groups;
};

// Rows per tile: the smallest of 16, 32, 64, 128 that holds the R rows, or 128 and several
// tiles. CTAs: one per SM, the row tiles side by side on the same keys; with
// more than 8 row tiles about two per SM instead, so that an uneven number of
// tiles costs less than the half-empty last wave.
TreePlan plan_tree(int64_t R) {
  const int n_sm = device_sm_count();
  const int64_t sms = n_sm > 0 ? n_sm : 148;
  TreePlan pl;
  pl.nr = R <= 16 ? 16 : R <= 32 ? 32 : R <= 64 ? 64 : kMaxRows;
  pl.rtiles = static_cast<int>(cdiv64(R, pl.nr));
  pl.groups = static_cast<int>(pl.rtiles <= 8 ? sms / pl.rtiles : cdiv64(2 * sms, pl.rtiles));
  if (pl.groups < 1) pl.groups = 1;
  return pl;
}

// Bytes of the parts' outputs and of all (one CTA per row tile: no pair is cut).
size_t part_bytes(const TreePlan& pl, int64_t D, size_t* o_bytes) {
  const size_t rows = pl.groups == 1 ? 0 : static_cast<size_t>(pl.rtiles) * pl.groups * 2 * pl.nr;
  *o_bytes = align256(rows * D * 4);
  return *o_bytes + align256(rows * 2 * 4) + 256;
}

bool map_keys(CUtensorMap* map, const mfa_tensor* t) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(t->D), static_cast<cuuint64_t>(t->N), static_cast<cuuint64_t>(t->H),
                        static_cast<cuuint64_t>(t->B)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(t->stride[2]) * 2, static_cast<cuuint64_t>(t->stride[1]) * 2,
                           static_cast<cuuint64_t>(t->stride[0]) * 2};
  cuuint32_t box[4] = {64, kKeys, 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, t->data, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NR>
mfa_status launch_tree(const CUtensorMap& mk, const CUtensorMap& mv, const TreeParams& p, cudaStream_t s) {
  using C = Cfg<D, NR>;
  static std::atomic<uint64_t> attr_devs{0};
  if (!ensure_smem_attr(reinterpret_cast<const void*>(mfa_tree_kernel<D, NR>), C::kBytes, attr_devs)) return MFA_ERR_CUDA;
  mfa_tree_kernel<D, NR><<<static_cast<unsigned>(p.rtiles) * p.groups, C::kThreads, C::kBytes, s>>>(mk, mv, p);
  if (cudaGetLastError() != cudaSuccess) return MFA_ERR_CUDA;
  if (p.groups > 1) {
    const int64_t pairs = static_cast<int64_t>(p.B) * p.Hkv;
    const int rows = p.R < NR ? p.R : NR;
    const int rpb = pairs * p.R <= 1024 ? 1 : 8;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(pairs), static_cast<unsigned>((rows + rpb - 1) / rpb * p.rtiles));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, mfa_tree_merge<D, NR>, p, rpb) != cudaSuccess) return MFA_ERR_CUDA;
  }
  return MFA_OK;
}

template <int D>
mfa_status launch_tree_rows(int nr, const CUtensorMap& mk, const CUtensorMap& mv, const TreeParams& p, cudaStream_t s) {
  switch (nr) {
    case 16: return launch_tree<D, 16>(mk, mv, p, s);
    case 32: return launch_tree<D, 32>(mk, mv, p, s);
    case 64: return launch_tree<D, 64>(mk, mv, p, s);
    default: return launch_tree<D, 128>(mk, mv, p, s);
  }
}

}  // namespace
}  // namespace mfa

extern "C" size_t mfa_tree_decode_workspace_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t T, int32_t D) {
  using namespace mfa;
  if (B < 0 || Hq <= 0 || Hkv <= 0 || T < 0 || Hq % Hkv || (D != 64 && D != 128 && D != 256)) return 0;
  if (B == 0 || T == 0) return 256;
  size_t o_bytes;
  return part_bytes(plan_tree(static_cast<int64_t>(T) * (Hq / Hkv)), D, &o_bytes);
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
  const int64_t R = q->N * (q->H / k->H);
  const TreePlan pl = plan_tree(R);
  size_t o_bytes;
  const size_t need = part_bytes(pl, q->D, &o_bytes);
  if (!workspace || workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
    return MFA_ERR_INVALID_ARG;
  CUtensorMap mk, mv;
  if (!map_keys(&mk, k) || !map_keys(&mv, v)) return MFA_ERR_CUDA;
  TreeParams p;
  p.B = static_cast<int32_t>(q->B); p.Hq = static_cast<int32_t>(q->H); p.Hkv = static_cast<int32_t>(k->H);
  p.G = static_cast<int32_t>(q->H / k->H); p.T = static_cast<int32_t>(q->N); p.N = static_cast<int32_t>(k->N);
  p.R = static_cast<int32_t>(R);
  p.rtiles = pl.rtiles; p.groups = pl.groups;
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(q->D)));
  p.q = static_cast<const __nv_bfloat16*>(q->data);
  for (int a = 0; a < 3; ++a) {
    p.qs[a] = q->stride[a]; p.os[a] = out->stride[a];
  }
  p.lens = lens; p.parents = parents;
  p.out = static_cast<__nv_bfloat16*>(out->data); p.lse = lse; p.err = dev_err;
  p.o_part = static_cast<float*>(workspace);
  p.ml_part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + o_bytes);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (q->D == 64) return launch_tree_rows<64>(pl.nr, mk, mv, p, s);
  if (q->D == 128) return launch_tree_rows<128>(pl.nr, mk, mv, p, s);
  return launch_tree_rows<256>(pl.nr, mk, mv, p, s);
}

// mfa_tree_decode: attention of a tree of drafted tokens over a cache.
//
// out[b, h, t] = sum_j p_j v_j with p = softmax over the keys j the row sees of
// q . k_j / sqrt(D): every key before lens[b], and of the drafted ones behind
// it node t itself and its ancestors. The R = T * G rows of a key/value head
// (row t * G + h') read the same keys, so K and V are read once for a tile of
// up to 128 rows; with more rows the CTAs of the row tiles walk the same keys side by
// side and share them in L2. Bound: HBM up to about 100 rows (8 x 8 lists of
// 31,000 keys of 256 columns, 16 rows each: 295 us, 7.0 TB/s), above them the softmax
// and its exchange with the products (8 x 8 lists of 25,000 keys of 128, 256
// rows each: 238 us, 713 TFLOP/s; 288 us where the power limit lowers the clock).
//
// Up to 64 rows (and for D = 256) the products are transposed, S^T = K Q^T and
// O^T += V^T P^T, so that the 128 rows of a tcgen05 MMA are 128 keys (or D
// columns) and its N is the number of query rows, 16, 32 or 64: a decoded token
// pays for 16 rows, not 128, and a thread holds the scores of ONE key for 16 rows. The
// running maximum of a row is shared by the threads through shared memory and
// only checked (one comparison chain and one vote per 128 keys, beside the
// exponentials); it moves when a score exceeds it by more than 8 (2^8 fits
// every type here), and the sums stay per thread until the end. P^T goes to
// shared memory as bf16 (the tensor core's input type; half a step of each
// weight), where it lies as the MMA's B operand wants it. More rows: see
// mfa_tree_rows_kernel.
//
// The tiles (128 keys) of all (batch, head) pairs are laid end to end and cut
// into equal ranges, one per CTA, from the lengths on the device: the grid
// does not depend on them. A pair met by one CTA is written directly; of a
// pair cut between CTAs each writes an unnormalised part (m, l, o), and a
// dependent launch merges them in a fixed order. The next pair's Q, K and V are
// loaded, and its first S computed, while a pair ends.
#include <cfloat>
#include <climits>
#include <cmath>
#include <cuda_bf16.h>

#include "cache.cuh"
#include "mfa_device.cuh"

namespace mfa {
namespace {

constexpr int kMaxRows = 128;        // query rows per row tile
constexpr int kSeenWords = MFA_TREE_MAX_NODES / 32;
constexpr float kLazy = 8.0f;        // a row's maximum moves when a score exceeds it by this (in powers of two)

struct TreeParams {
  int32_t B, Hq, Hkv, G, T, N, R;  // R = T * G rows per key/value head
  FastDiv by_g;
  int32_t rtiles, groups;          // row tiles; CTAs per row tile
  int32_t tile_t, parts;           // nodes per row tile; row tiles per node (1 unless G exceeds a tile)
  float scale_log2;
  int64_t os[3];
  const int32_t *lens, *parents;
  __nv_bfloat16* out;
  float *lse, *o_part, *ml_part;  // parts: [rtiles * groups][2][NR][D] and [..][NR][2] (m, l)
  int2* cut;                      // [rtiles][B][Hkv] a pair's first CTA, and how many it has
  uint32_t* err;
};

// Row tile rt: whole nodes, so that Q comes by TMA (a box of the group's heads by
// tile_t nodes), or part of one node's heads. Rows past the last one in Q's
// tile are zeros or other rows of Q.
struct RowTile {
  int row0, rows, node0, head0;  // first row, rows, first node and head
  __device__ __forceinline__ RowTile(const TreeParams& p, int rt, int nr) {
    if (p.parts == 1) {
      node0 = rt * p.tile_t;
      head0 = 0;
      rows = min(p.tile_t, p.T - node0) * p.G;
    } else {
      node0 = rt / p.parts;
      head0 = rt % p.parts * nr;
      rows = min(nr, p.G - head0);
    }
    row0 = node0 * p.G + head0;
  }
  __device__ __forceinline__ int last_node(const TreeParams& p) const { return p.parts == 1 ? min(node0 + p.tile_t, p.T) - 1 : node0; }
};

// By the CTA that has pair w's first tile: the CTAs that share the pair, for the merge. Those
// behind this one each take `per` places of it.
__device__ __forceinline__ void note_cut(const TreeParams& p, const Walk& w, int rt, int cta, int per) {
  p.cut[(static_cast<int64_t>(rt) * p.B + w.b) * p.Hkv + w.g] = make_int2(cta, 1 + (w.nt - w.t1 + per - 1) / per);
}

// Q of a row tile by TMA: its boxes of 64 columns.
template <int D, int NR>
__device__ __forceinline__ void load_q(const TreeParams& p, const CUtensorMap* tm_q, uint8_t* to, uint64_t* full, const RowTile& rows, int b, int g) {
  mbar_arrive_expect_tx(full, static_cast<uint32_t>(p.parts == 1 ? p.tile_t * p.G : NR) * 128u * (D / 64));
#pragma unroll
  for (int c = 0; c < D / 64; ++c) tma_load_4d(to + c * (NR * 128), tm_q, full, c * 64, g * p.G + rows.head0, rows.node0, b);
}

// ---------------------------------------------------------------------------
// Layout. K and V come in units of 128 keys x 128 columns (64 for D = 64), each
// through its own ring: a slot has one consumer (the S or the P.V warp), which
// waits for its phases in order, so a parity always names the phase meant.
// ---------------------------------------------------------------------------
template <int D, int NR>
struct Cfg {
  static constexpr int kCols = 16;                      // rows (registers) per softmax thread, as wide as the loads from TMEM
  static constexpr int kGroups = NR / kCols;            // groups of 4 softmax warps
  static constexpr int kSoftWarps = 4 * kGroups;
  static constexpr int kThreads = (kSoftWarps + 4) * 32;  // + S, P.V, TMA of K and V, TMA of Q
  static constexpr int kUnits = D == 256 ? 2 : 1;       // ring units of a K (or V) tile
  static constexpr int kUnit = (D == 64 ? 1 : 2) * kChunk;
  static constexpr int kPBytes = (NR + 63) / 64 * kChunk;
  static constexpr int kPBufs = D == 256 && NR == 64 ? 1 : 2;
  static constexpr int kRingK = D == 64 ? 4 : 2;
  static constexpr int kRingV = D == 64 ? 4 : 3;
  static constexpr int kRing = kRingK + kRingV;         // K's slots first
  static constexpr int kExtra = D == 256 ? 1 : D == 64 ? 4 : 2;  // see Line
  static constexpr int kQ = 0;                          // NR rows x 128 B per 64 columns
  static constexpr int kQBytes = NR * D * 2;
  static constexpr int kRing0 = (kQBytes + 1023) / 1024 * 1024;
  static constexpr int kP = kRing0 + kRing * kUnit;     // behind the ring: D = 64 reads one chunk past its last unit
  static constexpr int kMisc = kP + kPBufs * kPBytes;
  static constexpr int kBytes = kMisc + NR * 17 + 360;
  static constexpr int kO = 2 * NR;                     // TMEM columns: S0 [0, NR) S1 [NR, 2 NR) O [2 NR, (2 + kUnits) NR)
  static constexpr int kTmem = 4 * NR;
  static_assert(NR <= 64, "rows");
  static_assert(kBytes <= 232448, "shared memory");
  static_assert(kTmem <= 512, "TMEM columns");
};

__device__ __forceinline__ float warp_max(float x) {  // NaN is ignored unless all are
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Reduces v[c] over the warp's lanes: lane l ends with the result of column l / 2 in
// v[0], by halvings that hand half of the columns on.
template <typename Op>
__device__ __forceinline__ float warp_reduce_spread(float (&v)[16], int lane, Op op) {
#pragma unroll
  for (int w = 16, n = 8; w > 1; w >>= 1, n >>= 1) {
    const bool up = lane & w;
#pragma unroll
    for (int c = 0; c < n; ++c) {
      const float give = up ? v[c] : v[c + n], keep = up ? v[c + n] : v[c];
      v[c] = op(keep, __shfl_xor_sync(0xffffffffu, give, w));
    }
  }
  return v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}

// By the warp that issues P.V, before tile t's: V of a key that is not before
// the sequence's end must be finite, seen or not, as 0 * inf would reach every
// row. Rows of V that are not, and rows past the last node, become zeros; the rows of the output
// that see such a node become NaN in the epilogue, by the bits in bad (a tree) and *bad_min
// (a chain). Key r's columns are 128-byte rows of 64 columns in the U ring units `unit`.
// Returns how many steps of 16 keys the product has.
template <int D, int U>
__device__ __forceinline__ int clean_values(const TreeParams& p, const Walk& w, int t, int lane, uint32_t* bad, int* bad_min,
                                            uint8_t* const (&unit)[U]) {
  if (t == w.t0) {
    if (lane < kSeenWords) bad[lane] = 0u;
    if (lane == 0) *bad_min = INT_MAX;
    __syncwarp();
  }
  if (t * kKeys + kKeys <= w.len) return kKeys / 16;
  constexpr int kWide = D < 128 ? D / 8 : 16, kAtOnce = 32 / kWide;  // 16-byte units of a row in a ring unit; rows
  const int begin = max(w.len - t * kKeys, 0), end = min(min(w.len + p.T, p.N) - t * kKeys, kKeys);
  const int steps = (end + 15) / 16, c = lane % kWide;
  uint8_t* mine[U];
#pragma unroll
  for (int u = 0; u < U; ++u) mine[u] = unit[u] + (c >> 3) * kChunk + (c & 7) * 16;
#pragma unroll 4
  for (int r0 = begin; r0 < steps * 16; r0 += kAtOnce) {
    const int r = r0 + lane / kWide;
    uint32_t x = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint4 y = r < end ? *reinterpret_cast<const uint4*>(mine[u] + r * 128) : make_uint4(0u, 0u, 0u, 0u);
      // An exponent of ones carries into the sign's place.
      x |= ((y.x & 0x7f807f80u) + 0x00800080u) | ((y.y & 0x7f807f80u) + 0x00800080u) | ((y.z & 0x7f807f80u) + 0x00800080u) |
           ((y.w & 0x7f807f80u) + 0x00800080u);
    }
    x &= 0x80008000u;
    const unsigned lanes = __ballot_sync(0xffffffffu, x != 0);
    const bool broken = (lanes >> (lane / kWide * kWide) & ((1u << (kWide - 1)) * 2u - 1u)) != 0u;
    if (broken || (r >= end && r < steps * 16)) {
#pragma unroll
      for (int u = 0; u < U; ++u) *reinterpret_cast<uint4*>(mine[u] + r * 128) = make_uint4(0u, 0u, 0u, 0u);
    }
    if (broken && c == 0) {
      const int node = t * kKeys + r - w.len;
      if (p.parents) atomicOr(bad + (node >> 5), 1u << (node & 31));
      atomicMin(bad_min, node);
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
  return steps;
}

template <int D, int NR>
__global__ void __launch_bounds__(Cfg<D, NR>::kThreads, 1)
    mfa_tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TreeParams p) {
  using C = Cfg<D, NR>;
  constexpr int U = C::kUnits, RK = C::kRingK, RV = C::kRingV, RING = C::kRing, PB = C::kPBufs, W = C::kCols;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rt = blockIdx.x % p.rtiles, cta = blockIdx.x / p.rtiles;

  float* sNegM = reinterpret_cast<float*>(smem + C::kMisc);  // [NR] minus the row's maximum; 0 while it has none
  float* sDelta = sNegM + NR;                                // [NR] what the row's outputs are multiplied by
  float* sAlpha = sDelta + NR;                               // [NR] what its sums are multiplied by as its maximum moves
  float* sRed = sAlpha + NR;                                 // [NR] with sDelta and sAlpha: what warps 1 to 3 of a group hand to warp 0
  uint8_t* sSet = reinterpret_cast<uint8_t*>(sRed + NR);     // [NR] the row has a maximum
  uint32_t* sBad = reinterpret_cast<uint32_t*>(sSet + NR);   // [kSeenWords] a tree's nodes whose values are not finite,
  int* sBadMin = reinterpret_cast<int*>(sBad + kSeenWords);  // [2] a chain's first one (INT_MAX: none; a tree: any below that)
  uint64_t* bars = reinterpret_cast<uint64_t*>(sBadMin + 2);
  uint64_t* full = bars;               // [RING]
  uint64_t* empty = full + RING;       // [RING]
  uint64_t* q_full = empty + RING;     // Q of the next pair is in shared memory
  uint64_t* q_empty = q_full + 1;      // the pair's S are done
  uint64_t* s_full = q_empty + 1;      // [2]
  uint64_t* s_empty = s_full + 2;      // [2] read for the last time
  uint64_t* p_full = s_empty + 2;      // [PB]
  uint64_t* p_empty = p_full + 2;      // [PB] P.V done
  uint64_t* drain = p_empty + 2;       // [2]
  uint64_t* voted = drain + 2;         // [groups]
  int* sOver = reinterpret_cast<int*>(voted + 4);  // [groups][2] number + 1 of a tile that moves maxima
  volatile int* s_abort = reinterpret_cast<volatile int*>(sOver + 8);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(const_cast<int*>(s_abort) + 1);
  static_assert(40 + (2 * RING + 16) * 8 + 40 <= 360, "misc");

  // The merging kernel may be scheduled now: it waits for this grid to end.
  asm volatile("griddepcontrol.launch_dependents;");
  if (warp == C::kSoftWarps + 2 && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    for (int i = 0; i < RING; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], C::kSoftWarps);
      mbar_init(&p_full[i], C::kSoftWarps);
      mbar_init(&p_empty[i], 2);
      mbar_init(&drain[i], 1);
    }
    for (int i = 0; i < C::kGroups; ++i) {
      mbar_init(&voted[i], 4);
      sOver[2 * i] = sOver[2 * i + 1] = 0;
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    *s_abort = 0;
    fence_mbarrier_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const RowTile tile(p, rt, NR);
  const Line ln{p.lens, p.B, p.Hkv, p.N, tile.last_node(p), C::kExtra};
  const Start start = find_start(ln, cta, p.groups);
  if (start.b < 0) return;  // more CTAs than places
  Walk w(ln, start, p.groups);
  if (!w.more) return;      // none of them a tile
  const int per = places_per_cta(start.total, p.groups);
  const uint32_t ring = smem_u32(smem + C::kRing0);
  const int tile_fill = p.parts == 1 ? p.tile_t * p.G : NR;  // rows of Q's box
  // The TMA producer's state: K (and V) units issued; slots ever loaded, parity of the last load.
  uint32_t idx = 0, used = 0, phase = 0;
  // K and V of tile t; false when a wait ran out.
  auto load_tile = [&](int t) {
#pragma unroll
    for (int x = 0; x < 2 * U; ++x) {
      const bool isv = x >= U;
      const uint32_t u = x % U, at = idx + u, ring_n = isv ? RV : RK;
      const uint32_t slot = (isv ? RK : 0) + at % ring_n;
      if (at >= ring_n && !mbar_wait(&empty[slot], (at / ring_n - 1) & 1, s_abort)) return false;
      mbar_arrive_expect_tx(&full[slot], C::kUnit);
      uint8_t* dst = smem + C::kRing0 + slot * C::kUnit;
#pragma unroll
      for (int c = 0; c < C::kUnit / kChunk; ++c)
        tma_load_4d(dst + c * kChunk, isv ? &tm_v : &tm_k, &full[slot], u * 128 + c * 64, t * kKeys, w.g, w.b);
      used |= 1u << slot;
      phase = at / ring_n & 1 ? phase | 1u << slot : phase & ~(1u << slot);
    }
    idx += U;
    return true;
  };
  if (warp == C::kSoftWarps + 2 && lane == 0) {
    load_q<D, NR>(p, &tm_q, smem + C::kQ, q_full, tile, w.b, w.g);
    load_tile(w.t0);
  }
  // Rows of Q's buffer that no load fills.
  for (int i = threadIdx.x; i < (NR - tile_fill) * (D / 8); i += C::kThreads)
    *reinterpret_cast<uint4*>(smem + C::kQ + (i % (D / 8) >> 3) * (NR * 128) + (tile_fill + i / (D / 8)) * 128 + (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  if (warp == C::kSoftWarps) {
    tmem_alloc(s_tmem, C::kTmem);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  if (warp >= C::kSoftWarps) {
   if (warp == C::kSoftWarps + 2) {
    // =================== TMA producer ===================
    if (lane == 0) {
      bool ok = true;
      for (int t = w.t0 + 1; t < w.t1 && ok; ++t) ok = load_tile(t);
      while (ok && w.next(ln))
        for (int t = w.t0; t < w.t1 && ok; ++t) ok = load_tile(t);
      if (*s_abort) {
        // Loads in flight land before the CTA exits.
        volatile int no_abort = 0;
        for (int i = 0; i < RING; ++i)
          if (used >> i & 1) mbar_wait(&full[i], phase >> i & 1, &no_abort);
      }
    }
   } else if (warp == C::kSoftWarps + 3) {
    // =================== TMA of the next pairs' Q ===================
    if (lane == 0) {
      int seg = 0;  // of the last load
      while (w.next(ln) && mbar_wait(q_empty, seg & 1, s_abort)) {
        load_q<D, NR>(p, &tm_q, smem + C::kQ, q_full, tile, w.b, w.g);
        ++seg;
      }
      if (*s_abort) {
        volatile int no_abort = 0;
        mbar_wait(q_full, seg & 1, &no_abort);
      }
    }
   } else if (warp == C::kSoftWarps) {
    // =================== S^T = K Q^T ===================
    constexpr uint32_t idesc = idesc_keys(NR, false);
    const uint32_t q_addr = smem_u32(smem + C::kQ);
    bool ok = true;
    int n = 0, seg = 0;
    do {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(q_full, seg & 1, s_abort));
      for (int t = w.t0; t < w.t1 && ok; ++t, ++n) {
        const uint32_t first = static_cast<uint32_t>(n) * U;
        if (n >= 2 && !(ok = __all_sync(0xffffffffu, mbar_wait(&s_empty[n & 1], ((n >> 1) - 1) & 1, s_abort)))) break;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t slot = (first + u) % RK;
          if (!(ok = ok && __all_sync(0xffffffffu, mbar_wait(&full[slot], ((first + u) / RK) & 1, s_abort)))) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / U / 16; ++kk) {
            const uint32_t ka = ring + slot * C::kUnit + (kk >> 2) * kChunk + (kk & 3) * 32;
            const uint32_t qb = q_addr + (u * 2 + (kk >> 2)) * (NR * 128) + (kk & 3) * 32;
            umma_ss(tmem + (n & 1) * NR, sdesc_sw128_lo(ka, 16), sdesc_sw128_lo(qb, 16), idesc, u + kk > 0 ? 1u : 0u);
          }
          umma_commit(&empty[slot]);
        }
        umma_commit(&s_full[n & 1]);
      }
      umma_commit(q_empty);
      ++seg;
    } while (ok && w.next(ln));
    umma_commit(&drain[0]);
    volatile int no_abort = 0;
    mbar_wait(&drain[0], 0, &no_abort);
   } else if (warp == C::kSoftWarps + 1) {
    // =================== O^T += V^T P^T ===================
    constexpr uint32_t idesc = idesc_keys(NR, true);
    bool ok = true;
    int n = 0;
    do {
      for (int t = w.t0; t < w.t1 && ok; ++t, ++n) {
        const uint32_t first = static_cast<uint32_t>(n) * U;
        const uint32_t pb = sdesc_sw128_lo(smem_u32(smem + C::kP) + (n % PB) * C::kPBytes, kChunk);
        const bool draft = t * kKeys + kKeys > w.len;
        int steps = kKeys / 16;
        // V is cleaned while P is computed, but in a pair's first tile, whose P also says that
        // the last epilogue has read sBad.
        if (!draft || t == w.t0) ok = warp_wait(&p_full[n % PB], (n / PB) & 1, s_abort);
        if (ok && (draft || t == w.t0)) {
          uint8_t* unit[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const uint32_t slot = RK + (first + u) % RV;
            unit[u] = smem + C::kRing0 + slot * C::kUnit;
            ok = ok && warp_wait(&full[slot], ((first + u) / RV) & 1, s_abort);
          }
          if (ok) steps = clean_values<D, U>(p, w, t, lane, sBad, sBadMin, unit);
          if (ok && t != w.t0) ok = warp_wait(&p_full[n % PB], (n / PB) & 1, s_abort);
        }
        if (!ok) break;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t slot = RK + (first + u) % RV;
          if (!(ok = ok && __all_sync(0xffffffffu, mbar_wait(&full[slot], ((first + u) / RV) & 1, s_abort)))) break;
          tc_fence_after();
          const uint32_t va = sdesc_sw128_lo(ring + slot * C::kUnit, kChunk);
          const uint32_t more_o = t > w.t0 ? 1u : 0u, d_o = tmem + C::kO + u * NR;
          if (steps == kKeys / 16) {
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              umma_ss(d_o, va + kk * (16 * 128 / 16), pb + kk * (16 * 128 / 16), idesc, kk > 0 ? 1u : more_o);
          } else {
#pragma unroll 1
            for (int kk = 0; kk < steps; ++kk)
              umma_ss(d_o, va + kk * (16 * 128 / 16), pb + kk * (16 * 128 / 16), idesc, kk > 0 ? 1u : more_o);
          }
          umma_commit(&empty[slot]);
        }
        umma_commit(&p_empty[n % PB]);
        if (lane == 0) mbar_arrive(&p_empty[n % PB]);  // (orders sBad before the epilogue)
      }
    } while (ok && w.next(ln));
    umma_commit(&drain[1]);
    volatile int no_abort = 0;
    mbar_wait(&drain[1], 0, &no_abort);
   }
  } else {
    // =================== softmax and epilogue: a thread per key ===================
    // A failed wait raises *s_abort and the thread runs on (every later wait
    // then fails at once): the barriers below need all of the group's threads.
    const int grp = warp >> 2, quad = warp & 3;
    const int tid = quad * 32 + lane;           // key of the tile; column of D
    const uint32_t bar = 1 + grp;               // the group's named barrier
    constexpr uint32_t kAll = 1 + C::kGroups;   // all groups'
    const int col0 = grp * W;                   // its first row of the tile
    const uint32_t tm = tmem + (static_cast<uint32_t>(quad * 32) << 16) + col0;
    const int row0 = tile.row0 + col0;          // its first row of the pair
    const int rows = min(W, tile.rows - col0);  // real ones (may be <= 0)
    float* negM = sNegM + col0;
    float* delta = sDelta + col0;
    float* alpha = sAlpha + col0;
    // Row col0 + c's slot of warp `quad` (1 to 3).
    float* slot = (quad == 1 ? sRed : quad == 2 ? sDelta : sAlpha) + col0;
    const float* red = sRed + col0;
    int n = 0;
    uint32_t votes = 0;
    do {
      const int32_t* par = p.parents ? p.parents + static_cast<int64_t>(w.b) * p.T : nullptr;
      if (tid < W) {
        negM[tid] = 0.f;
        sSet[col0 + tid] = 0;
      }
      if (threadIdx.x == 0 && w.t0 == 0 && p.groups > 1) note_cut(p, w, rt, cta, per);
      if (rt == 0 && w.g == 0 && w.t0 == 0) {
        for (int t = threadIdx.x; t < (par ? p.T : 1); t += C::kSoftWarps * 32) {
          const uint32_t e = draft_errors(p.lens, p.parents, w.b, t, p.T, p.N);
          if (e) atomicOr(p.err, e);
        }
      }
      named_barrier(bar, 128);
      uint64_t l[W / 2];
#pragma unroll
      for (int c = 0; c < W / 2; ++c) l[c] = 0ull;

      for (int t = w.t0; t < w.t1; ++t, ++n) {
        const int base = t * kKeys;
        const uint32_t st = tm + (n & 1) * NR;  // the scores
        uint8_t* pbuf = smem + C::kP + (n % PB) * C::kPBytes;
        mbar_wait(&s_full[n & 1], (n >> 1) & 1, s_abort);
        tc_fence_after();
        const bool draft = base + kKeys > w.len;
        uint32_t see = ~0u;  // rows that see this thread's key, as bits
        if (draft) {
          // ---- a tile with drafted keys, or the last: who sees what ----
          const int j = base + tid, node = j - w.len;
          if (j >= min(w.len + p.T, p.N)) see = 0u;
          if (!par) {
            if (j >= w.len) see &= rows_from(node * p.G - row0);
          } else {
            // P's buffer is free (the wait passes while it was never used); its
            // slice of the group holds the parents and the nodes each row sees.
            mbar_wait(&p_empty[n % PB], ((n / PB) - 1) & 1, s_abort);
            int* sPar = reinterpret_cast<int*>(pbuf + grp * (C::kPBytes / C::kGroups));
            uint32_t* sSeen = reinterpret_cast<uint32_t*>(sPar + MFA_TREE_MAX_NODES);  // [W][kSeenWords]
            for (int i = tid; i < p.T; i += 128) sPar[i] = par[i];
            for (int i = tid; i < W * kSeenWords; i += 128) sSeen[i] = 0u;
            named_barrier(bar, 128);
            if (tid < rows && tid < W) {
              const int tt = p.by_g(row0 + tid);
              for (int a = sPar[tt] == -2 ? -1 : tt; a >= 0; a = tree_up(sPar, a))
                sSeen[tid * kSeenWords + (a >> 5)] |= 1u << (a & 31);
            }
            named_barrier(bar, 128);
            if (j >= w.len && see != 0u) {
              see = 0u;
#pragma unroll
              for (int c = 0; c < W; ++c) see |= ((sSeen[c * kSeenWords + (node >> 5)] >> (node & 31)) & 1u) << c;
            }
            named_barrier(kAll, C::kSoftWarps * 32);  // every group has looked: P may be written
          }
        }
        auto scores = [&](float (&y)[W]) {
          uint32_t r[W];
          tmem_ld_32x32b_x16(st, r);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < W; ++c) y[c] = __uint_as_float(r[c]);
          if (draft) {
#pragma unroll
            for (int c = 0; c < W; ++c)
              if (!(see >> c & 1)) y[c] = -INFINITY;
          }
        };
        // ---- weights 2^x of the scores x in powers of two relative to the rows'
        // maxima, and P in bf16 ----
        // A pair's first tile sets the maxima; a row may still have none in a
        // tile of drafted keys only. Otherwise they move when a score exceeds
        // one by more than kLazy: the warps vote on that while they compute the
        // weights, and compute them again where one says so.
        float x[W];
        bool renew = t == w.t0 || base >= w.len;
#pragma unroll 1
        for (bool again = renew;; again = true) {
          if (renew) {
            // Warp 3's slot is alpha, which the last tile may still be scaling by: the vote orders that,
            // the tree's table does, and a chain's tile of drafted keys, which has neither, does here.
            if (base >= w.len && t > w.t0 && !par) named_barrier(bar, 128);
            scores(x);
#pragma unroll
            for (int c = 0; c < W; ++c) x[c] = fmaf(x[c], p.scale_log2, negM[c]);
            float m = warp_reduce_spread(x, lane, [](float a, float b) { return fmaxf(a, b); });
            if (quad > 0) slot[lane / 2] = m;  // (two lanes write the same value)
            m = __shfl_sync(0xffffffffu, m, (lane & 15) * 2);
            named_barrier(bar, 128);
            bool moved = false;
            if (tid < W) {
              m = fmaxf(fmaxf(m, red[tid]), fmaxf(delta[tid], alpha[tid]));
              const bool set = sSet[col0 + tid] != 0;
              float d = 0.f;
              if (m > (set ? kLazy : -INFINITY)) {
                const float nm = negM[tid] - m;
                d = negM[tid] - nm;
                negM[tid] = nm;
                sSet[col0 + tid] = 1;
              } else if (!set) {
                sOver[2 * grp + (~n & 1)] = n + 2;  // every score -inf so far: the next tile sets the maximum
              }
              alpha[tid] = set ? ex2_approx(-d) : 1.f;  // a row without a maximum has no sums yet
              moved = set && d != 0.f;
            }
            if (vote_or(bar, 128, moved)) {
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
              for (int u = 0; u < U; ++u) {
                const uint32_t at = tm + C::kO + u * NR;
                uint32_t o[16];
                tmem_ld_32x32b_x16(at, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha[i]);
                tmem_st_32x32b_x16(at, o);
              }
              tmem_st_wait();
            }
          }
          scores(x);
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
          if (!again) {
            const bool over = __any_sync(0xffffffffu, fmaxf(mx[0], mx[1]) > kLazy);
            if (lane == 0) {
              if (over) sOver[2 * grp + (n & 1)] = n + 1;
              mbar_arrive(&voted[grp]);
            }
          }
          if (n >= PB) mbar_wait(&p_empty[n % PB], ((n / PB) - 1) & 1, s_abort);
          uint8_t* prow = pbuf + (col0 >> 6) * kChunk + tid * 128;
#pragma unroll
          for (int u = 0; u < W / 8; ++u) {
            uint32_t pk[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float& e0 = x[u * 8 + 2 * i];
              float& e1 = x[u * 8 + 2 * i + 1];
              e0 = ex2_approx(e0);
              e1 = ex2_approx(e1);
              pk[i] = pack_bf16x2(e0, e1);
            }
            *reinterpret_cast<uint4*>(prow + ((((col0 & 63) / 8 + u) ^ (tid & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
          if (again) break;
          mbar_wait(&voted[grp], votes & 1, s_abort);
          ++votes;
          renew = *reinterpret_cast<volatile int*>(&sOver[2 * grp + (n & 1)]) == n + 1;
          if (!renew) break;
        }
#pragma unroll
        for (int c = 0; c < W / 2; ++c) l[c] = f2_add(l[c], f2_pack(x[2 * c], x[2 * c + 1]));
        tc_fence_before();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&s_empty[n & 1]);
          mbar_arrive(&p_full[n % PB]);
        }
      }

      // ---- epilogue of the pair: its output, or this CTA's part of it ----
      const bool whole = w.t0 == 0 && w.t1 == w.nt;
      const int64_t part = (static_cast<int64_t>(blockIdx.x) * 2 + (w.t0 > 0 ? 0 : 1)) * NR + col0;
      float part_sum;
      named_barrier(bar, 128);  // the last tile's alpha has been read
      mbar_wait(&p_empty[(n - 1) % PB], ((n - 1) / PB) & 1, s_abort);  // O and sBad are complete
      tc_fence_after();
      {
        float v[W];
#pragma unroll
        for (int c = 0; c < W / 2; ++c) f2_unpack(l[c], v[2 * c], v[2 * c + 1]);
        part_sum = warp_reduce_spread(v, lane, [](float a, float b) { return a + b; });
        if (quad > 0) slot[lane / 2] = part_sum;
        part_sum = __shfl_sync(0xffffffffu, part_sum, (lane & 15) * 2);
      }
      named_barrier(bar, 128);
      if (tid < rows && tid < W) {
        const int tt = p.by_g(row0 + tid), h = w.g * p.G + row0 + tid - tt * p.G;
        const bool dead = par && par[tt] == -2;
        const float sum = dead ? 0.f : (part_sum + red[tid]) + (delta[tid] + alpha[tid]);
        const float m = -negM[tid];
        // Does the row see a node whose values are not finite? (Not dead: the row's way up is
        // the one its keys were masked by.)
        bool poison = *sBadMin <= tt;
        if (poison && par) {
          poison = false;
          for (int a = tt; a >= 0; a = tree_up(par, a)) poison |= sBad[a >> 5] >> (a & 31) & 1u;
        }
        // -1: no output. (A part without weights still makes a row that sees such a node NaN, as
        // the pair's sum does where it is not cut.)
        delta[tid] = sum == 0.f && (whole || dead || !poison) ? -1.f : (poison ? NAN : (whole ? 1.f / sum : 1.f));
        if (whole) {
          p.lse[(static_cast<int64_t>(w.b) * p.Hq + h) * p.T + tt] =
              sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.69314718055994530942f;
        } else {
          *reinterpret_cast<float2*>(p.ml_part + (part + tid) * 2) = make_float2(sum == 0.f ? -FLT_MAX : m, sum);
        }
        // Where the row goes, over what is no longer needed.
        const int64_t to = w.b * p.os[0] + h * p.os[1] + tt * p.os[2];
        reinterpret_cast<int*>(negM)[tid] = static_cast<int>(to);
        reinterpret_cast<int*>(alpha)[tid] = static_cast<int>(to >> 32);
      }
      named_barrier(bar, 128);
#pragma unroll 1
      for (int u = 0; u < U; ++u) {
        const int d = u * 128 + tid;
        if (rows <= 0) break;
        uint32_t o[16];
        tmem_ld_32x32b_x16(tm + C::kO + u * NR, o);
        tmem_ld_wait();
        if (d < D) {
          if (whole) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              if (i >= rows) break;
              const float f = delta[i];
              const int64_t to = static_cast<int64_t>(static_cast<uint32_t>(reinterpret_cast<const int*>(negM)[i])) |
                                 (static_cast<int64_t>(reinterpret_cast<const int*>(alpha)[i]) << 32);
              p.out[to + d] = __float2bfloat16_rn(f == -1.f ? 0.f : __uint_as_float(o[i]) * f);
            }
          } else {
            float* to = p.o_part + part * D + d;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              if (i >= rows) break;
              const float f = delta[i];
              to[i * D] = f == -1.f ? 0.f : __uint_as_float(o[i]) * f;
            }
          }
        }
      }
      tc_fence_before();
      named_barrier(bar, 128);  // what the next pair overwrites has been read
    } while (w.next(ln));
    if (*s_abort && threadIdx.x == 0) atomicOr(p.err, MFA_DEVERR_TIMEOUT);
  }
  __syncthreads();
  if (warp == C::kSoftWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// ---------------------------------------------------------------------------
// More than 64 rows (D up to 128): the rows as the MMA's 128, S = Q K^T and
// O += P V. With the keys as rows both operands of every product come from
// shared memory, 8 KB for each 128 x 128 x 16 product of 64 cycles, which with P's
// way through it and the loads' fills it (2,700 cycles per 128 rows and 128
// keys measured). Here P goes through tensor memory and halves that. Two groups of 128 threads, a
// thread per row, take turns on the tiles, each with its own S, running
// maximum, sum and output; the two are merged when the pair ends, as parts
// are. A group's S(n + 2) waits for its P.V(n), which has P in S's place, so the
// groups' softmaxes and products interleave.
// ---------------------------------------------------------------------------
template <int D>
struct RowCfg {
  static constexpr int kExtra = 10;  // (2 to 14 measured over 12 cases of 96 to 496 rows: within 3% from 7 on)
  static constexpr int kThreads = 384;                  // two softmax groups; MMA, TMA of K and V, TMA of Q, an idle one
  static constexpr int kRegsLow = 104, kRegsHigh = 200;  // 384 x 168 = 128 x 104 + 256 x 200
  static constexpr int kTile = D / 64 * kChunk;         // K or V of a tile
  static constexpr int kRing = D == 64 ? 5 : 3;         // tiles of each
  static constexpr int kQ = 0;                          // 128 rows x 128 B per 64 columns
  static constexpr int kK = kTile, kV = kK + kRing * kTile;
  static constexpr int kMisc = kV + kRing * kTile;
  static constexpr int kBytes = kMisc + 2 * 2 * 128 * 4 + MFA_TREE_MAX_NODES * 2 + 40 + (4 * kRing + 9) * 8 + 8;
  static constexpr int kO = 256;                        // TMEM columns: S0 [0, 128) S1 [128, 256) O0, O1 [256, 256 + 2 D)
  static_assert(128 * kRegsLow + 256 * kRegsHigh <= kThreads * 168, "register split");
  static_assert(kBytes <= 232448, "shared memory");
};

template <int D>
__global__ void __launch_bounds__(RowCfg<D>::kThreads, 1)
    mfa_tree_rows_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TreeParams p) {
  using C = RowCfg<D>;
  constexpr int RING = C::kRing, NR = 128;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rt = blockIdx.x % p.rtiles, cta = blockIdx.x / p.rtiles;

  float* sM = reinterpret_cast<float*>(smem + C::kMisc);       // [2][128] the groups' maxima and sums
  float* sL = sM + 2 * 128;
  int16_t* sPar = reinterpret_cast<int16_t*>(sL + 2 * 128);    // [T] a tree's parents (those past int16 as -3: they end the way up)
  uint32_t* sBad = reinterpret_cast<uint32_t*>(sPar + MFA_TREE_MAX_NODES);  // as in mfa_tree_kernel
  int* sBadMin = reinterpret_cast<int*>(sBad + kSeenWords);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(sBadMin + 2);  // [RING]
  uint64_t* k_empty = k_full + RING;
  uint64_t* v_full = k_empty + RING;
  uint64_t* v_empty = v_full + RING;
  uint64_t* q_full = v_empty + RING;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_empty + 1;  // [2]
  uint64_t* p_full = s_full + 2;   // [2]
  uint64_t* pv_done = p_full + 2;  // [2] a group's last P.V of a pair is done
  uint64_t* drain = pv_done + 2;
  volatile int* s_abort = reinterpret_cast<volatile int*>(drain + 1);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(const_cast<int*>(s_abort) + 1);

  asm volatile("griddepcontrol.launch_dependents;");
  if (warp == 10 && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    for (int i = 0; i < RING; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 2);
    }
    mbar_init(drain, 1);
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    *s_abort = 0;
    fence_mbarrier_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const RowTile tile(p, rt, NR);
  const Line ln{p.lens, p.B, p.Hkv, p.N, tile.last_node(p), C::kExtra};
  const Start start = find_start(ln, cta, p.groups);
  if (start.b < 0) return;  // more CTAs than places
  Walk w(ln, start, p.groups);
  if (!w.more) return;      // none of them a tile
  const int per = places_per_cta(start.total, p.groups);
  int parent = 0;  // of node threadIdx.x
  auto fetch_parent = [&](int b) {
    if (p.parents && static_cast<int>(threadIdx.x) < p.T) parent = p.parents[static_cast<int64_t>(b) * p.T + threadIdx.x];
  };
  if (warp < 8) fetch_parent(w.b);
  int tiles = 0, loads_k = 0;  // the producer's: tiles loaded, K loads
  auto load_tile = [&](int t) {
    const int slot = tiles % RING, round = tiles / RING;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (round > 0 && !mbar_wait(x ? &v_empty[slot] : &k_empty[slot], (round - 1) & 1, s_abort)) return false;
      uint64_t* full = x ? &v_full[slot] : &k_full[slot];
      mbar_arrive_expect_tx(full, C::kTile);
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        tma_load_4d(smem + (x ? C::kV : C::kK) + slot * C::kTile + c * kChunk, x ? &tm_v : &tm_k, full, c * 64, t * kKeys, w.g, w.b);
      if (x == 0) ++loads_k;
    }
    ++tiles;
    return true;
  };
  if (warp == 10 && lane == 0) {
    load_q<D, NR>(p, &tm_q, smem + C::kQ, q_full, tile, w.b, w.g);
    load_tile(w.t0);
  }
  // Rows of Q's buffer that no load fills.
  const int tile_fill = p.parts == 1 ? p.tile_t * p.G : NR;
  for (int i = threadIdx.x; i < (NR - tile_fill) * (D / 8); i += C::kThreads)
    *reinterpret_cast<uint4*>(smem + C::kQ + (i % (D / 8) >> 3) * (NR * 128) + (tile_fill + i / (D / 8)) * 128 + (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  if (warp == 8) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsLow));
    if (warp == 10) {
      // =================== TMA producer ===================
      if (lane == 0) {
        bool ok = true;
        for (int t = w.t0 + 1; t < w.t1 && ok; ++t) ok = load_tile(t);
        while (ok && w.next(ln))
          for (int t = w.t0; t < w.t1 && ok; ++t) ok = load_tile(t);
        if (*s_abort) {
          // Loads in flight land before the CTA exits.
          volatile int no_abort = 0;
          for (int j = loads_k > RING ? loads_k - RING : 0; j < loads_k; ++j) mbar_wait(&k_full[j % RING], (j / RING) & 1, &no_abort);
          for (int j = tiles > RING ? tiles - RING : 0; j < tiles; ++j) mbar_wait(&v_full[j % RING], (j / RING) & 1, &no_abort);
        }
      }
    } else if (warp == 11) {
      // =================== TMA of the next pairs' Q ===================
      if (lane == 0) {
        int seg = 0;  // of the last load
        while (w.next(ln) && mbar_wait(q_empty, seg & 1, s_abort)) {
          load_q<D, NR>(p, &tm_q, smem + C::kQ, q_full, tile, w.b, w.g);
          ++seg;
        }
        if (*s_abort) {
          volatile int no_abort = 0;
          mbar_wait(q_full, seg & 1, &no_abort);
        }
      }
    } else if (warp == 8) {
      // =================== S = Q K^T, O += P V ===================
      // P.V(n) and S(n + 2), which overwrites its P, go out together: products of one thread
      // run in order. S of the next pair follows the pair's last P.V, as it waits for the next Q.
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, kKeys, false), idesc_o = idesc_bf16_f32(128, D, true);
      const uint32_t q_addr = smem_u32(smem + C::kQ), k_addr = smem_u32(smem + C::kK), v_addr = smem_u32(smem + C::kV);
      bool ok = true;
      int n = 0, seg = 0;  // the next P.V's tile; pairs begun
      auto issue_s = [&](int k) {
        const int slot = k % RING;
        if (!__all_sync(0xffffffffu, mbar_wait(&k_full[slot], (k / RING) & 1, s_abort))) return false;
        tc_fence_after();
        const uint32_t kb = k_addr + slot * C::kTile;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * kChunk + (kk & 3) * 32;
          umma_ss(tmem + (k & 1) * 128, sdesc_sw128_lo(q_addr + off, 16), sdesc_sw128_lo(kb + off, 16), idesc_s, kk > 0 ? 1u : 0u);
        }
        umma_commit(&s_full[k & 1]);
        umma_commit(&k_empty[slot]);
        return true;
      };
      do {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(q_full, seg & 1, s_abort));
        ok = ok && issue_s(n);
        if (w.t1 - w.t0 > 1) ok = ok && issue_s(n + 1);
        for (int t = w.t0; t < w.t1 && ok; ++t, ++n) {
          const int slot = n % RING;
          // (A pair's first P also says that the last epilogue has read sBad.)
          ok = __all_sync(0xffffffffu, mbar_wait(&v_full[slot], (n / RING) & 1, s_abort));
          if (t == w.t0) ok = ok && __all_sync(0xffffffffu, mbar_wait(&p_full[n & 1], (n >> 1) & 1, s_abort));
          if (!ok) break;
          uint8_t* unit[1] = {smem + C::kV + slot * C::kTile};
          const int steps = clean_values<D, 1>(p, w, t, lane, sBad, sBadMin, unit);
          if (t != w.t0 && !(ok = __all_sync(0xffffffffu, mbar_wait(&p_full[n & 1], (n >> 1) & 1, s_abort)))) break;
          tc_fence_after();
          const uint32_t vd = sdesc_sw128_lo(v_addr + slot * C::kTile, kChunk);
          const uint32_t a_p = tmem + (n & 1) * 128, d_o = tmem + C::kO + (n & 1) * D;
          const uint32_t more_o = t >= w.t0 + 2 ? 1u : 0u;
          // (Unrolled for whole tiles: a step behind a condition takes twice its 64 cycles to issue.)
          if (steps == kKeys / 16) {
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk) umma_ts(d_o, a_p + kk * 8, vd + kk * (16 * 128 / 16), idesc_o, kk > 0 ? 1u : more_o);
          } else {
#pragma unroll 1
            for (int kk = 0; kk < steps; ++kk) umma_ts(d_o, a_p + kk * 8, vd + kk * (16 * 128 / 16), idesc_o, kk > 0 ? 1u : more_o);
          }
          umma_commit(&v_empty[slot]);
          if (t + 2 < w.t1) {
            ok = issue_s(n + 2);
          } else {
            // The group's last of the pair: its epilogue waits for it.
            umma_commit(&pv_done[n & 1]);
            if (lane == 0) mbar_arrive(&pv_done[n & 1]);  // (orders sBad before the epilogue)
          }
        }
        umma_commit(q_empty);  // (after the pair's last S)
        ++seg;
      } while (ok && w.next(ln));
      umma_commit(drain);
      volatile int no_abort = 0;
      mbar_wait(drain, 0, &no_abort);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsHigh));
    // =================== softmax and epilogue: a thread per row ===================
    // (A failed wait raises *s_abort and the thread runs on, as in mfa_tree_kernel.)
    const int grp = warp >> 2, quad = warp & 3;
    const int r = quad * 32 + lane, row = tile.row0 + r;  // the thread's row of the tile, of the pair
    const bool real = r < tile.rows;
    const int node = real ? p.by_g(row) : 0, head = row - node * p.G;
    const uint32_t tm = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    int n = 0;  // tiles of the CTA before the pair's first
    uint32_t lasts = 0;  // of the group's last P.V of a pair
    do {
      const int32_t* par = p.parents ? p.parents + static_cast<int64_t>(w.b) * p.T : nullptr;
      if (par) sPar[threadIdx.x] = static_cast<int16_t>(parent < -2 || parent > INT16_MAX ? -3 : parent);
      if (threadIdx.x == 0 && w.t0 == 0 && p.groups > 1) note_cut(p, w, rt, cta, per);
      if (rt == 0 && w.g == 0 && w.t0 == 0) {
        for (int t = threadIdx.x; t < (par ? p.T : 1); t += 256) {
          const uint32_t e = draft_errors(p.lens, p.parents, w.b, t, p.T, p.N);
          if (e) atomicOr(p.err, e);
        }
      }
      if (par) named_barrier(1, 256);
      const bool dead = par && sPar[node] == -2;
      float m = -INFINITY, l = 0.f;
      const int count = w.t1 - w.t0;
      for (int i = (n & 1) == grp ? 0 : 1; i < count; i += 2) {
        const int k = n + i, base = (w.t0 + i) * kKeys;  // the tile's number in the CTA, its first key
        mbar_wait(&s_full[grp], (k >> 1) & 1, s_abort);
        tc_fence_after();
        float x[kKeys];
        {
          uint32_t y[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(tm + grp * 128 + c * 32, y[c]);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < kKeys; ++c) x[c] = __uint_as_float(y[c >> 5][c & 31]);
        }
        if (base + kKeys > w.len) {
          // ---- a tile with drafted keys, or the last: the keys the row sees, as bits ----
          const int own = w.len - base;  // drafted keys begin here
          uint32_t see[4];
          if (!par) {
            const int hi = min(own + node, p.N - 1 - base);  // the last one seen
#pragma unroll
            for (int c = 0; c < 4; ++c) see[c] = ~rows_from(hi + 1 - c * 32);
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) see[c] = ~rows_from(own - c * 32);
            for (int a = dead ? -1 : node; a >= 0; a = tree_up(sPar, a)) {
              const int at = own + a;
              if (at < p.N - base) {
#pragma unroll
                for (int c = 0; c < 4; ++c) see[c] |= (at >> 5) == c ? 1u << (at & 31) : 0u;
              }
            }
          }
#pragma unroll
          for (int c = 0; c < kKeys; ++c)
            if (!(see[c >> 5] >> (c & 31) & 1)) x[c] = -INFINITY;
        }
        // The weights are computed relative to the maximum so far while the tile's own is found:
        // it seldom moves (a group's first tile finds it first). Where one does, the
        // row's sums shrink and the warp computes the tile's weights again.
        uint64_t sum[2];
        bool again = i < 2;
#pragma unroll 1
        while (true) {
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          if (again) {
#pragma unroll
            for (int c = 0; c < kKeys; c += 8) {
#pragma unroll
              for (int y = 0; y < 4; ++y) mx[y] = fmax3(mx[y], x[c + 2 * y], x[c + 2 * y + 1]);
            }
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
            const bool need = top > m + kLazy;
            const float m_new = need ? top : m;
            if (i >= 2) {
              // O holds every P.V of the group before this tile's: S(k) went out after P.V(k - 2).
              const float alpha = need ? ex2_approx(m - m_new) : 1.f;  // (m = -inf: 0, and the sums are 0)
              l *= alpha;
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(tm + C::kO + grp * D + c, o);
                tmem_ld_wait();
#pragma unroll
                for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * alpha);
                tmem_st_32x32b_x32(tm + C::kO + grp * D + c, o);
              }
            }
            m = m_new;
          }
          const float m_use = m == -INFINITY ? 0.f : m;
          const uint64_t sc2 = f2_pack(p.scale_log2, p.scale_log2), nm2 = f2_pack(-m_use, -m_use);
          sum[0] = sum[1] = 0ull;
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            uint32_t pk[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const int y = h * 32 + 2 * c;
              float a, b;
              f2_unpack(f2_fma(f2_pack(x[y], x[y + 1]), sc2, nm2), a, b);
              a = ex2_approx(a);
              b = ex2_approx(b);
              mx[c & 3] = fmax3(mx[c & 3], x[y], x[y + 1]);
              sum[c & 1] = f2_add(sum[c & 1], f2_pack(a, b));
              pk[c] = pack_bf16x2(a, b);
            }
            tmem_st_32x32b_x16(tm + grp * 128 + h * 16, pk);
          }
          if (again) break;
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
          if (!__any_sync(0xffffffffu, top > m + kLazy)) break;
          again = true;
        }
        float a, b;
        f2_unpack(f2_add(sum[0], sum[1]), a, b);
        l += a + b;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[grp]);
      }
      Walk nx = w;
      const bool more = nx.next(ln);
      if (more) fetch_parent(nx.b);

      // ---- epilogue of the pair: merge the groups ----
      const int end = n + count;
      if (count > ((n & 1) == grp ? 0 : 1)) {  // the group had a tile
        mbar_wait(&pv_done[grp], lasts & 1, s_abort);
        ++lasts;
        tc_fence_after();
      }
      sM[grp * 128 + r] = m;
      sL[grp * 128 + r] = l;
      named_barrier(1, 256);
      tc_fence_after();
      {
        const float m0 = sM[r], m1 = sM[128 + r], l0 = sL[r], l1 = sL[128 + r];
        const float M = fmaxf(m0, m1);  // (-inf: no key seen, or only NaN scores)
        const float M_use = M == -INFINITY ? 0.f : M;
        const float f0 = m0 == -INFINITY ? 1.f : ex2_approx(m0 - M_use), f1 = m1 == -INFINITY ? 1.f : ex2_approx(m1 - M_use);
        const bool has0 = l0 != 0.f, has1 = l1 != 0.f;  // (a group without one may hold anything in O)
        const float sum = dead ? 0.f : (has0 ? l0 * f0 : 0.f) + (has1 ? l1 * f1 : 0.f);
        const bool whole = w.t0 == 0 && w.t1 == w.nt, any = real && sum != 0.f;
        bool poison = *sBadMin <= node;
        if (poison && par) {
          poison = false;
          for (int x = node; x >= 0; x = tree_up(sPar, x)) poison |= sBad[x >> 5] >> (x & 31) & 1u;
        }
        const float g = poison ? NAN : whole ? 1.f / sum : 1.f;
        const float g0 = f0 * g, g1 = f1 * g;
        const float none = poison && !whole && !dead ? NAN : 0.f;  // (as in mfa_tree_kernel)
        const int64_t part = (static_cast<int64_t>(blockIdx.x) * 2 + (w.t0 > 0 ? 0 : 1)) * NR + r;
        const int h = w.g * p.G + head;
        if (real && grp == 0) {
          if (whole)
            p.lse[(static_cast<int64_t>(w.b) * p.Hq + h) * p.T + node] = any ? (M_use + log2f(sum)) * 0.69314718055994530942f : -INFINITY;
          else
            *reinterpret_cast<float2*>(p.ml_part + part * 2) = make_float2(any ? M_use : -FLT_MAX, sum);
        }
        // Group g writes columns [g D / 2, (g + 1) D / 2).
        __nv_bfloat16* to = p.out + w.b * p.os[0] + h * p.os[1] + node * p.os[2];
        float* part_to = p.o_part + part * D;
#pragma unroll 1
        for (int c = grp * (D / 2); c < (grp + 1) * (D / 2); c += 16) {
          uint32_t o0[16], o1[16];
          tmem_ld_32x32b_x16(tm + C::kO + c, o0);
          tmem_ld_32x32b_x16(tm + C::kO + D + c, o1);
          tmem_ld_wait();
          float y[16];
#pragma unroll
          for (int u = 0; u < 16; ++u) {
            y[u] = has0 ? __uint_as_float(o0[u]) * g0 : 0.f;
            if (has1) y[u] = fmaf(__uint_as_float(o1[u]), g1, y[u]);
            if (!any) y[u] = none;
          }
          if (real) {
            if (whole) {
#pragma unroll
              for (int u = 0; u < 2; ++u)
                reinterpret_cast<uint4*>(to + c)[u] = make_uint4(pack_bf16x2(y[8 * u], y[8 * u + 1]), pack_bf16x2(y[8 * u + 2], y[8 * u + 3]),
                                                                 pack_bf16x2(y[8 * u + 4], y[8 * u + 5]), pack_bf16x2(y[8 * u + 6], y[8 * u + 7]));
            } else {
#pragma unroll
              for (int u = 0; u < 4; ++u)
                reinterpret_cast<float4*>(part_to + c)[u] = make_float4(y[4 * u], y[4 * u + 1], y[4 * u + 2], y[4 * u + 3]);
            }
          }
        }
      }
      tc_fence_before();
      named_barrier(1, 256);  // O, sM, sL, sPar have been read
      n = end;
      w = nx;
      if (!more) break;
    } while (true);
    if (*s_abort && threadIdx.x == 0) atomicOr(p.err, MFA_DEVERR_TIMEOUT);
  }
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// Merges the parts of every pair that was cut: with M = max m_s, out = sum o_s
// 2^(m_s - M) / sum l_s 2^(m_s - M). A part without a visible key has
// m = -FLT_MAX, l = 0, o = 0 (never -inf - -inf); all such: out = 0, lse = -inf.
// A warp takes a row, a lane D / 32 of its columns and, for M and the
// weights, every 32nd part: two rounds of loads. With few rows a block takes one
// row and its WS warps share the parts: 8 warps while all rows are resident at
// once (5 blocks per SM), 4 up to 12 rows per SM. (8 lists of 8000 keys, D = 128: 104 rows
// 18.0 us with 4 against 19.9 with 8 and 23.9 with a warp per row; 4 rows 9.2 with
// 8, 9.5 with 4; 2048 rows of 128 lists of 4000 49.3 with 4, 47.3 with a warp.)
// ---------------------------------------------------------------------------
constexpr int kMergeWarps = 8;

template <int D, int NR, int WS>
__global__ void __launch_bounds__((WS > 1 ? WS : kMergeWarps) * 32) mfa_tree_merge(const __grid_constant__ TreeParams p) {
  constexpr int E = D / 32;
  constexpr bool SPLIT = WS > 1;
  __shared__ float so[WS][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rt = blockIdx.y % p.rtiles;
  const int r = SPLIT ? blockIdx.y / p.rtiles : blockIdx.y / p.rtiles * kMergeWarps + warp;  // row of the row tile
  const int b = blockIdx.x / p.Hkv, g = blockIdx.x % p.Hkv;
  asm volatile("griddepcontrol.launch_dependents;");
  const RowTile tile(p, rt, NR);
  if (r >= tile.rows) return;  // (SPLIT: the whole block)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int2 cut = p.cut[static_cast<int64_t>(rt) * p.B * p.Hkv + blockIdx.x];
  const int c0 = cut.x, ns = cut.y;
  if (ns == 1) return;  // written by its only CTA
  // Part s of the row: the first CTA met the pair's first tile (its second slot), the
  // others begin inside it.
  auto at = [&](int s) {
    const int64_t c = c0 + s;
    return ((c * p.rtiles + rt) * 2 + (s > 0 ? 0 : 1)) * NR + r;
  };
  float M = -FLT_MAX;
  for (int s = lane; s < ns; s += 32) M = fmaxf(M, p.ml_part[at(s) * 2]);
  M = warp_max(M);
  float l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int s0 = 0; s0 < ns; s0 += 32) {
    float f = 0.f;
    if (s0 + lane < ns) {
      const float2 ml = *reinterpret_cast<const float2*>(p.ml_part + at(s0 + lane) * 2);
      f = ex2_approx(ml.x - M);
      l = fmaf(f, ml.y, l);
    }
    const int hi = min(32, ns - s0);
#pragma unroll 8
    for (int s = SPLIT ? warp : 0; s < hi; s += WS) {
      const float fs = __shfl_sync(0xffffffffu, f, s);
      const float* y = p.o_part + at(s0 + s) * D + lane * E;
      if constexpr (E == 2) {
        const float2 v = *reinterpret_cast<const float2*>(y);
        o[0] = fmaf(fs, v.x, o[0]); o[1] = fmaf(fs, v.y, o[1]);
      } else {
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          const float4 v = *reinterpret_cast<const float4*>(y + e);
          o[e] = fmaf(fs, v.x, o[e]); o[e + 1] = fmaf(fs, v.y, o[e + 1]);
          o[e + 2] = fmaf(fs, v.z, o[e + 2]); o[e + 3] = fmaf(fs, v.w, o[e + 3]);
        }
      }
    }
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
  if constexpr (SPLIT) {
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int x = 1; x < WS; ++x) o[e] += so[x][lane * E + e];
  }
  const int row = tile.row0 + r, t = p.by_g(row), h = g * p.G + row - t * p.G;
  const bool has = l != 0.f;
  const float inv = has ? 1.f / l : 0.f;
  uint32_t* to = reinterpret_cast<uint32_t*>(p.out + b * p.os[0] + h * p.os[1] + t * p.os[2] + lane * E);
  uint32_t y[E / 2];
#pragma unroll
  for (int e = 0; e < E / 2; ++e) y[e] = has ? pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv) : 0u;
  if constexpr (E == 2) *to = y[0];
  else if constexpr (E == 4) *reinterpret_cast<uint2*>(to) = make_uint2(y[0], y[1]);
  else *reinterpret_cast<uint4*>(to) = make_uint4(y[0], y[1], y[2], y[3]);
  if (lane == 0)
    p.lse[(static_cast<int64_t>(b) * p.Hq + h) * p.T + t] = has ? (M + log2f(l)) * 0.69314718055994530942f : -INFINITY;
}

// ---- host ----

struct TreePlan {
  int nr, rtiles, groups, tile_t, parts;
};

int64_t sm_count() {
  const int n = device_sm_count();
  return n > 0 ? n : 148;
}

// Rows per tile: the smallest of 16, 32, 64, 128 (D = 256: 64) that holds the
// T nodes' rows, or the largest and several tiles of whole nodes (of parts of one node's
// heads where G exceeds a tile). CTAs: one per SM, the row tiles side by side
// on the same keys. With more than 8 row tiles that could leave a quarter of the SMs idle
// (38 x 3 of 148), so that each gets its part of two CTAs per SM, rounded up: 9 x 33,
// 16 x 19 or 32 x 10 on 148 SMs, of which the few past 296 run in a third wave.
TreePlan plan_tree(int64_t T, int64_t G, int64_t D) {
  const int64_t sms = sm_count(), R = T * G;
  TreePlan pl;
  pl.nr = R <= 16 ? 16 : R <= 32 ? 32 : R <= 64 || D == 256 ? 64 : kMaxRows;
  pl.parts = static_cast<int>(cdiv64(G, pl.nr));
  pl.tile_t = pl.parts > 1 ? 1 : static_cast<int>(T < pl.nr / G ? T : pl.nr / G);
  pl.rtiles = static_cast<int>(pl.parts > 1 ? T * pl.parts : cdiv64(T, pl.tile_t));
  pl.groups = static_cast<int>(pl.rtiles <= 8 ? sms / pl.rtiles : cdiv64(2 * sms, pl.rtiles));
  if (pl.groups < 1) pl.groups = 1;
  return pl;
}

// Bytes of the parts' outputs, of their (m, l) and of all (one CTA per row tile: no pair is cut).
struct TreeSpace {
  size_t o, ml, all;
};
TreeSpace tree_space(const TreePlan& pl, int64_t D, int64_t pairs) {
  if (pl.groups == 1) return {0, 0, 256};
  const size_t rows = static_cast<size_t>(pl.rtiles) * pl.groups * 2 * pl.nr;
  const size_t o = align256(rows * D * 4), ml = align256(rows * 2 * 4);
  return {o, ml, o + ml + align256(static_cast<size_t>(pl.rtiles) * pairs * sizeof(int2))};
}

// The tensor map of q: boxes of 64 columns x the heads of a group x the nodes of a row tile.
bool map_queries(CUtensorMap* map, const mfa_tensor* q, const TreePlan& pl, int64_t G) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(q->D), static_cast<cuuint64_t>(q->H), static_cast<cuuint64_t>(q->N),
                        static_cast<cuuint64_t>(q->B)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(q->stride[1]) * 2, static_cast<cuuint64_t>(q->stride[2]) * 2,
                           static_cast<cuuint64_t>(q->stride[0]) * 2};
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(pl.parts > 1 ? pl.nr : G), static_cast<cuuint32_t>(pl.tile_t), 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, q->data, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NR, typename K>
mfa_status launch_tree(K kernel, int threads, int bytes, std::atomic<uint64_t>& attr_devs, const CUtensorMap& mq, const CUtensorMap& mk,
                       const CUtensorMap& mv, const TreeParams& p, cudaStream_t s) {
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kernel), bytes, attr_devs)) return MFA_ERR_CUDA;
  if (!launch_after(kernel, dim3(static_cast<unsigned>(p.rtiles) * p.groups), threads, bytes, s, mq, mk, mv, p)) return MFA_ERR_CUDA;
  if (p.groups > 1) {
    const int64_t pairs = static_cast<int64_t>(p.B) * p.Hkv;
    const int rows = p.parts > 1 ? NR : p.tile_t * p.G;  // of a tile
    const int64_t sms = sm_count();
    const int ws = pairs * p.R <= 5 * sms ? 8 : pairs * p.R <= 12 * sms ? 4 : 1;
    const dim3 grid(static_cast<unsigned>(pairs), static_cast<unsigned>((ws > 1 ? rows : cdiv64(rows, kMergeWarps)) * p.rtiles));
    auto* merge = ws == 8 ? mfa_tree_merge<D, NR, 8> : ws == 4 ? mfa_tree_merge<D, NR, 4> : mfa_tree_merge<D, NR, 1>;
    if (!launch_after(merge, grid, (ws > 1 ? ws : kMergeWarps) * 32, 0, s, p)) return MFA_ERR_CUDA;
  }
  return MFA_OK;
}

template <int D, int NR>
mfa_status launch_keys(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const TreeParams& p, cudaStream_t s) {
  using C = Cfg<D, NR>;
  static std::atomic<uint64_t> attr_devs{0};
  return launch_tree<D, NR>(mfa_tree_kernel<D, NR>, C::kThreads, C::kBytes, attr_devs, mq, mk, mv, p, s);
}

template <int D>
mfa_status launch_rows(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const TreeParams& p, cudaStream_t s) {
  using C = RowCfg<D>;
  static std::atomic<uint64_t> attr_devs{0};
  return launch_tree<D, 128>(mfa_tree_rows_kernel<D>, C::kThreads, C::kBytes, attr_devs, mq, mk, mv, p, s);
}

template <int D>
mfa_status launch_tree_rows(int nr, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const TreeParams& p, cudaStream_t s) {
  switch (nr) {
    case 16: return launch_keys<D, 16>(mq, mk, mv, p, s);
    case 32: return launch_keys<D, 32>(mq, mk, mv, p, s);
    case 64: return launch_keys<D, 64>(mq, mk, mv, p, s);
    default:
      if constexpr (D == 256) return MFA_ERR_UNSUPPORTED;  // plan_tree gives no such tile
      else return launch_rows<D>(mq, mk, mv, p, s);
  }
}

}  // namespace
}  // namespace mfa

extern "C" size_t mfa_tree_decode_workspace_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t T, int32_t D) {
  using namespace mfa;
  if (B < 0 || Hq <= 0 || Hkv <= 0 || T < 0 || Hq % Hkv || (D != 64 && D != 128 && D != 256)) return 0;
  if (B == 0 || T == 0) return 256;
  return tree_space(plan_tree(T, Hq / Hkv, D), D, static_cast<int64_t>(B) * Hkv).all;
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
  const TreePlan pl = plan_tree(q->N, q->H / k->H, q->D);
  const TreeSpace sp = tree_space(pl, q->D, k->B * k->H);
  if (!workspace || workspace_bytes < sp.all || reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
    return MFA_ERR_INVALID_ARG;
  CUtensorMap mq, mk, mv;
  if (!map_queries(&mq, q, pl, q->H / k->H) || !map_keys(&mk, k) || !map_keys(&mv, v)) return MFA_ERR_CUDA;
  TreeParams p;
  p.B = static_cast<int32_t>(q->B); p.Hq = static_cast<int32_t>(q->H); p.Hkv = static_cast<int32_t>(k->H);
  p.G = static_cast<int32_t>(q->H / k->H); p.T = static_cast<int32_t>(q->N); p.N = static_cast<int32_t>(k->N);
  p.R = static_cast<int32_t>(R);
  p.by_g.set(static_cast<uint32_t>(p.G));
  p.rtiles = pl.rtiles; p.groups = pl.groups; p.tile_t = pl.tile_t; p.parts = pl.parts;
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(q->D)));
  for (int a = 0; a < 3; ++a) p.os[a] = out->stride[a];
  p.lens = lens; p.parents = parents;
  p.out = static_cast<__nv_bfloat16*>(out->data); p.lse = lse; p.err = dev_err;
  p.o_part = static_cast<float*>(workspace);
  p.ml_part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + sp.o);
  p.cut = reinterpret_cast<int2*>(static_cast<uint8_t*>(workspace) + sp.o + sp.ml);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (q->D == 64) return launch_tree_rows<64>(pl.nr, mq, mk, mv, p, s);
  if (q->D == 128) return launch_tree_rows<128>(pl.nr, mq, mk, mv, p, s);
  return launch_tree_rows<256>(pl.nr, mq, mk, mv, p, s);
}

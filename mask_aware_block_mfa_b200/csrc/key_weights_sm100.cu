// mfa_key_weights: the attention weight every cached key got from a call's
// rows, w[b, g, j] = decay * w_in + sum over heads h of group g and rows t that
// see j of row_scale[t] * exp(q_ht . k_j / sqrt(D) - lse_ht).
//
// S^T = K Q^T on tcgen05 as in tree decode, 128 keys by the R = T * G rows of a
// key/value head, so that a thread holds one key's scores for 16 to 128 rows at
// a time and adds its own key's weight: no sum crosses threads but the one
// over row tiles. K is read once for up to 256 rows (128 at D = 256), and nothing
// else of size is. Bound: HBM (2 D bytes per key) up to about 150 rows, beyond them the
// 16 exponentials per clock of an SM. (4 x 8 lists of 32768 keys, 128 rows: 52
// us, 5.3 TB/s, 64 us at the 1.5 GHz of the power limit; 8 x 8 lists of 22,000, 64 rows: 62 us, 6.0 TB/s.)
//
// What a row adds to every score, -lse and the logarithm of its scale's size, would cost
// each thread a shared-memory read per row (as much of the SM's time as the
// exponentials); it comes out of the tensor core instead, as 16 more products
// per score: ones for the key times the constant in three bf16 parts, which
// hold a float32's 24 bits, added after the D others so that they are not rounded at its size.
#include <cmath>
#include <cuda_bf16.h>

#include "cache.cuh"
#include "mfa_device.cuh"

namespace mfa {
namespace {

constexpr int kGroups = 4;                        // softmax groups of 128 threads
constexpr int kSoftThreads = kGroups * 128;
constexpr int kThreads = kSoftThreads + 64;       // + the MMA and the TMA warp
constexpr int kMaxRing = 12;
constexpr int kSmem = 232448;

struct KeyWeightParams {
  int32_t B, Hq, Hkv, G, T, N, R;
  FastDiv by_g;
  int32_t row0, qtiles;          // rows of this pass: row0 .., in qtiles (1 or 2) tiles of NR
  int32_t ring, words, ctas;     // K units; 32-bit words of a row's nodes; CTAs of the line
  float scale_log2, decay, unscale;  // unscale: 1 / scale_log2
  const __nv_bfloat16* q;
  int64_t qs[3];
  const float *lse, *row_scale, *w_in;
  const int32_t *lens, *parents;
  float* w_out;
  uint32_t* err;
};

template <int D, int NR>
struct Cfg {
  static constexpr int kUnits = D == 256 ? 2 : 1;   // ring units of a K tile
  static constexpr int kUnit = (D == 64 ? 1 : 2) * kChunk;
  static constexpr int kQTile = NR * D * 2;         // NR rows x 128 B per 64 columns
  static constexpr int kExtra = D == 256 ? 4 : D == 64 ? 12 : 8;
  static constexpr int kBufs = NR <= 64 ? 2 * kGroups : kGroups;  // TMEM buffers of S, one or two for each group
  static constexpr int kBars = 2 * kMaxRing + 1 + 2 * kBufs + 1;
  // Bytes besides the ring (first) and Q (next): constants and ones, signs, partial sums, who sees what, barriers.
  static constexpr int rest(int qtiles, int T, int words) {
    return kChunk + qtiles * NR * 4 + 2 * kSoftThreads * 4 + 32 + (words > 0 ? T * 4 + T * words * 4 : 0) + 16 + kBars * 8 + 16;
  }
  // K units beside them.
  static constexpr int units(int qtiles, int T, int words) { return (kSmem - qtiles * kQTile - rest(qtiles, T, words)) / kUnit; }
  // Two row tiles in one pass: up to 64 rows are one tile, and at D = 256 two of 128 (64 KB each) leave no ring
  // of two K tiles. More than two would not help: with two the exponentials already take longer than K's next read.
  static constexpr bool kTwo = NR == 128 && D < 256;
  static_assert(units(kTwo ? 2 : 1, MFA_TREE_MAX_NODES, MFA_TREE_MAX_NODES / 32) >= 2 * kUnits, "ring");
};

template <int D, int NR>
__global__ void __launch_bounds__(kThreads, 1)
    mfa_key_weights_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ KeyWeightParams p) {
  using C = Cfg<D, NR>;
  constexpr int U = C::kUnits, X = NR < 32 ? NR : 32;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int qtiles = C::kTwo ? p.qtiles : 1;
  uint8_t* sQ = smem + p.ring * C::kUnit;                              // [qtiles]
  // 128-byte rows: the rows' constants, 32 bytes for each row tile, and from byte 96 on the keys' ones, 1 1 1 0 ..
  uint8_t* sConst = sQ + qtiles * C::kQTile;                           // [128]
  float* sSign = reinterpret_cast<float*>(sConst + kChunk);            // [qtiles * NR] of the row's scale; 0: it is left out
  float* sPart = sSign + qtiles * NR;                                  // [2][kGroups][128]
  uint32_t* sActive = reinterpret_cast<uint32_t*>(sPart + 2 * kSoftThreads);  // [8] bits: the row counts
  uint64_t* full = reinterpret_cast<uint64_t*>(sActive + 8);           // [ring]
  uint64_t* empty = full + kMaxRing;
  uint64_t* q_full = empty + kMaxRing;
  uint64_t* s_full = q_full + 1;           // [kBufs]
  uint64_t* s_empty = s_full + C::kBufs;   // [kBufs]
  uint64_t* drain = s_empty + C::kBufs;
  volatile int* s_abort = reinterpret_cast<volatile int*>(drain + 1);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(const_cast<int*>(s_abort) + 1);
  int* sPar = reinterpret_cast<int*>(s_tmem + 1);                      // [T] the tree
  uint32_t* sSeen = reinterpret_cast<uint32_t*>(sPar + p.T);           // [T][words] the nodes each one sees

  asm volatile("griddepcontrol.launch_dependents;");
  if (warp == kGroups * 4 + 1 && lane == 0) {
    tma_prefetch_desc(&tm_k);
    for (int i = 0; i < p.ring; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::kBufs; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 4);
    }
    mbar_init(q_full, kSoftThreads);
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_mbarrier_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Line ln{p.lens, p.B, p.Hkv, p.N, p.T - 1, C::kExtra};
  const Start start = find_start(ln, blockIdx.x, p.ctas);
  if (start.b < 0) return;  // more CTAs than places
  Walk w(ln, start, p.ctas);
  if (!w.more) return;      // none of them a tile
  // What a pair's rows need from memory, fetched together: a thread's row (its
  // lse, scale and parent) and its part of the first kBatch steps of Q.
  constexpr int kStep = kSoftThreads / (D / 8), kBatch = NR < kStep ? 1 : NR / kStep < 4 ? NR / kStep : 4;
  const int qu = threadIdx.x % (D / 8), qr = threadIdx.x / (D / 8);
  struct {
    float lse, scale;
    int up;
    uint4 q[kBatch];
  } pre;
  auto fetch_q = [&](int i0) {
    const __nv_bfloat16* src = p.q + w.b * p.qs[0] + static_cast<int64_t>(w.g) * p.G * p.qs[1] + qu * 8;
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      const int row = min(p.row0 + i0 + y * kStep, p.R - 1), t = p.by_g(row), h = row - t * p.G;
      pre.q[y] = *reinterpret_cast<const uint4*>(src + h * p.qs[1] + t * p.qs[2]);
    }
  };
  auto fetch = [&]() {
    const int row = min(p.row0 + static_cast<int>(threadIdx.x), p.R - 1), t = p.by_g(row), h = w.g * p.G + row - t * p.G;
    pre.lse = p.lse[(static_cast<int64_t>(w.b) * p.Hq + h) * p.T + t];
    pre.scale = p.row_scale ? p.row_scale[static_cast<int64_t>(w.b) * p.T + t] : 1.f;
    pre.up = p.parents ? p.parents[static_cast<int64_t>(w.b) * p.T + t] : 0;
    fetch_q(qr);
  };
  if (threadIdx.x < kSoftThreads) fetch();
  int slot = 0, round = 0;  // the TMA producer's and the MMA issuer's: of the next unit
  // K of tile t; false when a wait ran out.
  auto load_tile = [&](int t) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (round > 0 && !mbar_wait(&empty[slot], (round - 1) & 1, s_abort)) return false;
      mbar_arrive_expect_tx(&full[slot], C::kUnit);
#pragma unroll
      for (int c = 0; c < C::kUnit / kChunk; ++c)
        tma_load_4d(smem + slot * C::kUnit + c * kChunk, &tm_k, &full[slot], u * 128 + c * 64, t * kKeys, w.g, w.b);
      if (++slot == p.ring) {
        slot = 0;
        ++round;
      }
    }
    return true;
  };
  if (warp == kGroups * 4 + 1 && lane == 0) load_tile(w.t0);
  if (warp == kGroups * 4) {
    tmem_alloc(s_tmem, C::kBufs * NR);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  if (warp == kGroups * 4 + 1) {
    // =================== TMA producer ===================
    if (lane == 0) {
      bool ok = true;
      for (int t = w.t0 + 1; t < w.t1 && ok; ++t) ok = load_tile(t);
      while (ok && w.next(ln))
        for (int t = w.t0; t < w.t1 && ok; ++t) ok = load_tile(t);
      if (*s_abort) {
        // Loads in flight land before the CTA exits.
        volatile int no_abort = 0;
        for (int i = 0; i < p.ring; ++i) {
          const int r = i < slot ? round : round - 1;  // the slot's last load
          if (r >= 0) mbar_wait(&full[i], r & 1, &no_abort);
        }
      }
    }
  } else if (warp == kGroups * 4) {
    // =================== S^T = K Q^T ===================
    // Item i = tile * qtiles + row tile goes to buffer i % kBufs and group i % 4.
    constexpr uint32_t idesc = idesc_keys(NR, false);
    const uint32_t ring = smem_u32(smem), q_addr = smem_u32(sQ);
    bool ok = true;
    uint32_t item = 0;
    int seg = 0;
    do {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(q_full, seg & 1, s_abort));
      for (int t = w.t0; t < w.t1 && ok; ++t) {
        for (int rt = 0; rt < qtiles; ++rt, ++item) {
          // The K units, and the buffer as its last sums were read (at once for the first uses: their phase is before the first).
          const int buf = item % C::kBufs;
          const uint32_t free = (item / C::kBufs + 1) & 1;
          int s2 = slot, r2 = round;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            ok = ok && (u == 0 ? warp_wait2(&full[s2], r2 & 1, &s_empty[buf], free, s_abort) : warp_wait(&full[s2], r2 & 1, s_abort));
            if (++s2 == p.ring) {
              s2 = 0;
              ++r2;
            }
          }
          if (!ok) break;
          tc_fence_after();
          s2 = slot;
#pragma unroll
          for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int kk = 0; kk < D / U / 16; ++kk) {
              const uint32_t ka = ring + s2 * C::kUnit + (kk >> 2) * kChunk + (kk & 3) * 32;
              const uint32_t qb = q_addr + rt * C::kQTile + (u * 2 + (kk >> 2)) * (NR * 128) + (kk & 3) * 32;
              umma_ss(tmem + buf * NR, sdesc_sw128_lo(ka, 16), sdesc_sw128_lo(qb, 16), idesc, u + kk > 0 ? 1u : 0u);
            }
            if (++s2 == p.ring) s2 = 0;
          }
          umma_ss(tmem + buf * NR, sdesc_sw128_lo(smem_u32(sConst) + 96, 16), sdesc_sw128_lo(smem_u32(sConst) + rt * 32, 16), idesc, 1u);
          umma_commit(&s_full[buf]);  // (the tile's last group hands the K units back)
        }
        if (!ok) break;
        slot += U;
        if (slot >= p.ring) {
          slot -= p.ring;
          ++round;
        }
      }
      ++seg;
    } while (ok && w.next(ln));
    umma_commit(drain);
    volatile int no_abort = 0;
    mbar_wait(drain, 0, &no_abort);
  } else {
    // =================== weights: a thread per key ===================
    // A failed wait raises *s_abort and the thread runs on (every later wait
    // then fails at once): the barriers below need all threads.
    const int grp = warp >> 2, tid = threadIdx.x & 127;
    const int rt = grp & (qtiles - 1), nn = kGroups / qtiles;  // the group's row tile; tiles in flight
    const uint32_t tm = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    for (int i = threadIdx.x; i < kKeys * 2; i += kSoftThreads) {
      const int r = i >> 1, u = i & 1;
      *reinterpret_cast<uint4*>(sConst + r * 128 + (((6 + u) ^ (r & 7)) << 4)) =
          u == 0 ? make_uint4(0x3f803f80u, 0x3f80u, 0u, 0u) : make_uint4(0u, 0u, 0u, 0u);
    }
    int n = 0;           // tiles of the CTA so far
    int k = 0;           // of them the group's
    do {
      const int32_t* par = p.parents ? p.parents + static_cast<int64_t>(w.b) * p.T : nullptr;
      float sign;  // of the thread's row's scale
      // ---- the pair's rows (all of the last pair's S and sums are done) ----
      // Rows that count for nothing, whatever they hold, become Q = 0 with a constant that
      // no exponential survives.
      {
        const int i = threadIdx.x, r = i % NR, q = i / NR;
        const bool real = i < qtiles * NR;
        float c = -1e30f;
        sign = 0.f;
        if (real && p.row0 + i < p.R && pre.scale != 0.f && pre.lse != -INFINITY && pre.up != -2) {
          sign = pre.scale < 0.f ? -1.f : 1.f;
          c = (log2f(fabsf(pre.scale)) - pre.lse * 1.4426950408889634f) * p.unscale;  // in the scores' unit
        }
        const unsigned active = __ballot_sync(0xffffffffu, sign != 0.f);
        if (lane == 0 && real) sActive[warp] = active;
        if (real) {
          sSign[i] = sign;
          uint32_t part[3];
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const __nv_bfloat16 y = __float2bfloat16_rn(c);
            part[k] = __bfloat16_as_ushort(y);
            c = isfinite(__bfloat162float(y)) ? c - __bfloat162float(y) : 0.f;
          }
          uint8_t* to = sConst + r * 128;
          *reinterpret_cast<uint4*>(to + (((2 * q) ^ (r & 7)) << 4)) = make_uint4(part[0] | part[1] << 16, part[2], 0u, 0u);
          *reinterpret_cast<uint4*>(to + (((2 * q + 1) ^ (r & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      if (par && w.t1 * kKeys > w.len)
        for (int i = threadIdx.x; i < p.T; i += kSoftThreads) sPar[i] = par[i];
      if (p.row0 == 0 && w.g == 0 && w.t0 == 0) {
        for (int t = threadIdx.x; t < (par ? p.T : 1); t += kSoftThreads) {
          const uint32_t e = draft_errors(p.lens, p.parents, w.b, t, p.T, p.N);
          if (e) atomicOr(p.err, e);
        }
      }
      const bool minus = vote_or(1, kSoftThreads, sign < 0.f);  // a row of the pair has a negative scale
      if (par && w.t1 * kKeys > w.len) {
        for (int t = threadIdx.x; t < p.T; t += kSoftThreads) {
          for (int x = 0; x < p.words; ++x) sSeen[t * p.words + x] = 0u;
          for (int a = sPar[t] == -2 ? -1 : t; a >= 0; a = tree_up(sPar, a)) sSeen[t * p.words + (a >> 5)] |= 1u << (a & 31);
        }
      }
      for (int i0 = qr; i0 < qtiles * NR; i0 += kBatch * kStep) {
        if (i0 != qr) fetch_q(i0);
#pragma unroll
        for (int y = 0; y < kBatch; ++y) {
          const int i = i0 + y * kStep, r = i % NR;
          if (i >= qtiles * NR) break;
          if (sSign[i] == 0.f) pre.q[y] = make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(sQ + (i / NR) * C::kQTile + (qu >> 3) * (NR * 128) + r * 128 + (((qu & 7) ^ (r & 7)) << 4)) = pre.q[y];
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(q_full);
      named_barrier(1, kSoftThreads);  // sSeen is complete

      const int64_t out0 = (static_cast<int64_t>(w.b) * p.Hkv + w.g) * p.N;
      const int end = min(w.len + p.T, p.N);
      for (int t = w.t0; t < w.t1; ++t, ++n) {
        if (n % nn != grp / qtiles) continue;
        const int j = t * kKeys + tid, node = j - w.len;
        const bool mine = rt == 0 && j < end, add = p.w_in != nullptr && p.decay != 0.f;
        float old = 0.f;
        if (mine && add) old = p.w_in[out0 + j];
        uint64_t acc[2] = {0ull, 0ull};
        constexpr int kEach = C::kBufs / kGroups;
        const int buf = grp + k % kEach * kGroups;
        const uint32_t st = tm + buf * NR;
        mbar_wait(&s_full[buf], (k / kEach) & 1, s_abort);
        tc_fence_after();
        // S of the tile's last row tile is done, and so those before it: K may be overwritten.
        if (rt == qtiles - 1 && tid < U) mbar_arrive(&empty[(n * U + tid) % p.ring]);
        const uint64_t sc2 = f2_pack(p.scale_log2, p.scale_log2);
        bool plain = t * kKeys + kKeys <= w.len && !minus;
        if (plain) {
#pragma unroll
          for (int c = 0; c < NR; c += X) {
            uint32_t x[X];
            if constexpr (X == 16) tmem_ld_32x32b_x16(st + c, x);
            else tmem_ld_32x32b_x32(st + c, x);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < X; i += 2) {
              float a, b;
              f2_unpack(f2_mul(f2_pack(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), sc2), a, b);
              acc[(i >> 1) & 1] = f2_add(acc[(i >> 1) & 1], f2_pack(ex2_approx(a), ex2_approx(b)));
            }
          }
          // An infinity in a key makes the rows left out NaN (their Q is 0): do those keys with the rows that count.
          float a, b;
          f2_unpack(f2_add(acc[0], acc[1]), a, b);
          plain = !__any_sync(0xffffffffu, isnan(a + b));
        }
        if (!plain) {
          // Negative scales, drafted keys or infinities: a thread leaves out the rows that do not see its key.
          float sum = 0.f;
          acc[0] = acc[1] = 0ull;
#pragma unroll 1
          for (int c = 0; c < NR; c += X) {
            const int first = p.row0 + rt * NR + c;
            uint32_t see = (sActive[(rt * NR + c) >> 5] >> (c & 31)) & (X == 32 ? ~0u : (1u << X) - 1u);
            if (j >= w.len) see = j < end ? see & (par ? rows_seeing<X>(sSeen, p.words, node, first, p.G, p.by_g, p.T) : rows_from(node * p.G - first)) : 0u;
            uint32_t x[X];
            if constexpr (X == 16) tmem_ld_32x32b_x16(st + c, x);
            else tmem_ld_32x32b_x32(st + c, x);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < X; ++i) x[i] = see >> i & 1 ? x[i] : 0xff800000u;
            if (minus) {
#pragma unroll
              for (int i = 0; i < X; ++i) sum = fmaf(ex2_approx(__uint_as_float(x[i]) * p.scale_log2), sSign[rt * NR + c + i], sum);
            } else {
#pragma unroll
              for (int i = 0; i < X; i += 2) {
                float a, b;
                f2_unpack(f2_mul(f2_pack(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), sc2), a, b);
                acc[(i >> 1) & 1] = f2_add(acc[(i >> 1) & 1], f2_pack(ex2_approx(a), ex2_approx(b)));
              }
            }
          }
          acc[0] = f2_add(acc[0], f2_pack(sum, 0.f));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[buf]);
        const uint64_t both = f2_add(acc[0], acc[1]);
        float lo, hi;
        f2_unpack(both, lo, hi);
        float sum = lo + hi;
        if (qtiles > 1) {
          // The row tiles' sums, in their order. (The barrier of the next tile is
          // passed only once these have been read: two buffers suffice.)
          float* part = sPart + (k & 1) * kSoftThreads;
          if (rt > 0) part[grp * 128 + tid] = sum;
          named_barrier(2 + grp / 2, 256);
          if (rt == 0) sum += part[(grp + 1) * 128 + tid];
        }
        if (mine) p.w_out[out0 + j] = add ? fmaf(p.decay, old, sum) : sum;
        ++k;
      }
      if (w.next(ln)) fetch();  // the next pair's
      named_barrier(1, kSoftThreads);  // every sum of the pair is done
    } while (w.more);
    if (*s_abort && threadIdx.x == 0) atomicOr(p.err, MFA_DEVERR_TIMEOUT);
  }
  __syncthreads();
  if (warp == kGroups * 4) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kBufs * NR);
  }
}

// ---- host ----

template <int D, int NR>
mfa_status launch_weights(const CUtensorMap& mk, KeyWeightParams p, cudaStream_t s) {
  using C = Cfg<D, NR>;
  static std::atomic<uint64_t> attr_devs{0};
  if (!ensure_smem_attr(reinterpret_cast<const void*>(mfa_key_weights_kernel<D, NR>), kSmem, attr_devs)) return MFA_ERR_CUDA;
  p.words = p.parents ? (p.T + 31) / 32 : 0;
  const int sms = device_sm_count();
  p.ctas = sms > 0 ? sms : 148;
  for (p.row0 = 0; p.row0 < p.R; p.row0 += p.qtiles * NR) {
    p.qtiles = C::kTwo && p.R - p.row0 > NR ? 2 : 1;
    p.ring = C::units(p.qtiles, p.T, p.words);
    if (p.ring > kMaxRing) p.ring = kMaxRing;
    const int bytes = p.ring * C::kUnit + p.qtiles * C::kQTile + C::rest(p.qtiles, p.T, p.words);
    if (!launch_after(mfa_key_weights_kernel<D, NR>, dim3(p.ctas), kThreads, bytes, s, mk, p)) return MFA_ERR_CUDA;
    // Later rows add to what this pass wrote.
    p.w_in = p.w_out;
    p.decay = 1.f;
  }
  return MFA_OK;
}

template <int D>
mfa_status launch_weights_rows(const CUtensorMap& mk, const KeyWeightParams& p, cudaStream_t s) {
  if (p.R <= 16) return launch_weights<D, 16>(mk, p, s);
  if (p.R <= 32) return launch_weights<D, 32>(mk, p, s);
  if (p.R <= 64) return launch_weights<D, 64>(mk, p, s);
  return launch_weights<D, 128>(mk, p, s);
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
  CUtensorMap mk;
  if (!map_keys(&mk, k)) return MFA_ERR_CUDA;
  KeyWeightParams p;
  p.B = static_cast<int32_t>(q->B); p.Hq = static_cast<int32_t>(q->H); p.Hkv = static_cast<int32_t>(k->H);
  p.G = static_cast<int32_t>(q->H / k->H); p.T = static_cast<int32_t>(q->N); p.N = static_cast<int32_t>(k->N);
  p.R = p.T * p.G;
  p.by_g.set(static_cast<uint32_t>(p.G));
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(q->D)));
  p.unscale = static_cast<float>(std::sqrt(static_cast<double>(q->D)) / 1.4426950408889634);
  p.decay = decay;
  p.q = static_cast<const __nv_bfloat16*>(q->data);
  for (int a = 0; a < 3; ++a) p.qs[a] = q->stride[a];
  p.lse = lse; p.row_scale = row_scale; p.w_in = weights_in; p.w_out = weights_out;
  p.lens = lens; p.parents = parents; p.err = dev_err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (q->D == 64) return launch_weights_rows<64>(mk, p, s);
  if (q->D == 128) return launch_weights_rows<128>(mk, p, s);
  return launch_weights_rows<256>(mk, p, s);
}

// Cross attention: segments of queries against segments of an encoder's
// states, of other lengths, and its gradients.
//
// For segment s with queries Q and keys and values K, V of one head (query
// head h reads key head h / (H / H_kv)):
//   S = Q K^T / sqrt(d_h),  P = softmax(S),  O = P V,  lse = log sum exp S;
// a segment without keys gives O = 0 and lse = -inf.  Backward:
//   D = rowsum(dO * O),  dP = dO V^T,  dS = P * (dP - D),
//   dV = P^T dO,  dK = dS^T Q / sqrt(d_h),  dQ = dS K / sqrt(d_h),
// with P = exp(S - lse), and dK, dV summed over the query heads that share a
// key head.
//
// cross_fwd_kernel<DH>  persistent, one CTA of 16 warps per SM.  A unit is two
//   128-row query tiles (A, B) of one (segment, key head): with r = H / H_kv
//   query heads to a key head a tile holds 128 / r tokens of all r heads
//   (one TMA box of 64 columns x r heads x 128 / r tokens), so that K and V are
//   read once for all of them.
//   warp 0  TMA of the K and V tiles (128 keys)
//   warp 3  walks the units and loads their query tiles
//   warp 1  tcgen05.mma: PV_A(j), S_A(j+1), PV_B(j), S_B(j+1); the next unit's
//           first S follows its last PV without a gap
//   warp 2  zeroes the rows of a V tile between the segment's last key and the
//           next multiple of 16 (the product runs in steps of 16 keys; a row of
//           another segment may hold NaN, and 0 * NaN is NaN)
//   warps 4-7, 8-11  softmax of tile A, B, one row per thread, half a row in
//           registers at a time: S is read from TMEM for the maximum and (its
//           second half again) for the exponentials, P is written over it in
//           bf16 and is the A operand of PV
//   warps 12-15  epilogue of both tiles: O / l from TMEM through 4 KB of shared
//           memory per warp to 128-byte row pieces.  Prompts are short: with 512
//           keys a unit has four steps, and an epilogue inside the softmax warps
//           would take as long as two of them.
// Measured at 187,200 x 512 keys, 12 heads of 128 channels: 0.55 to 0.57 ms,
// 1.05 PFLOP/s (0.63 of the measured cuBLAS burst; 0.67 ms in a long run under
// the power cap); of 64 channels 0.46 to 0.48 ms; x 128 keys of 128: 0.24 to
// 0.25 ms, 4.7 TB/s, near HBM's rate.  With long prompts no unit is full: a step
// of two query tiles and 128 keys takes 3,990 cycles, of which the products are
// 51 % (29 % at 64 channels) and the exponentials 52 % (57 %), instructions issue
// in 43 %, and 7 % of instruction fetches miss.  Softmax and products take turns
// more than they overlap; which wait makes up the rest is not measured.
// With few units the key range is split over CTAs, which write O / l and (l, m)
// in fp32, and cross_join_kernel joins them.
// How P keeps clear of infinities at scores of any size: P_factors in ptx.cuh.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "cross.cuh"

namespace moga {
namespace {

template <int C>
__device__ __forceinline__ void store_row(void* base, int64_t at, int lane, const float (&x)[C], float f) {
  __nv_bfloat16* p = static_cast<__nv_bfloat16*>(base) + at + lane * C;
#pragma unroll
  for (int i = 0; i < C; ++i) p[i] = __float2bfloat16(x[i] * f);
}

template <int DH>
struct XPlan {
  static constexpr int kStages = DH == 64 ? 4 : 2;
  static constexpr int kChunk = kTile * 128;         // bytes of 64 columns of a tile
  static constexpr int kTileBytes = kTile * DH * 2;
  static constexpr int kQ = 0;                       // tiles A, B
  static constexpr int kK = 2 * kTileBytes;
  static constexpr int kV = kK + kStages * kTileBytes;
  static constexpr int kStage = kV + kStages * kTileBytes;  // epilogue: 4 KB per warp
  static constexpr int kStat = kStage + 4 * 4096;    // [2 parities][2 tiles][128] of (l, m)
  static constexpr int kBar = kStat + 2 * 2 * kTile * 8;
  static constexpr int kFeed = kBar + 512;           // ring of units
  static constexpr int kBytes = kFeed + kFeedSlots * 32 + 1024;
  static_assert(kBytes <= 232448, "shared memory");
};


struct XMaps {
  CUtensorMap q, k, v;
  XView qv, kv, vv;
};

// kOne: units with one query tile take turns in both S buffers.  For calls of
// few rows a segment: 77 queries x 187,200 keys 272 -> 237 us; elsewhere the
// code it adds costs 4 %.
template <int DH, bool kOne>
__global__ void __launch_bounds__(kXThreads, 1)
cross_fwd_kernel(const __grid_constant__ XMaps m, const CrossArgs a, const XGrid xg, float* part_o, float2* part_lm,
                 int withhold, int* status, unsigned long long wait_ns) {
  using P = XPlan<DH>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + P::kBar);
  uint64_t* q_full = bars;                     // [2]
  uint64_t* q_empty = bars + 2;                // [2]
  // [3]: S computed, P written (O rescaled), of tile A, of B, and of A in B's
  // columns (a unit with one tile).  The last has barriers of its own: every
  // barrier is followed by one role through all its phases, or a wait's
  // parity could stand for the phase before.
  uint64_t* s_full = bars + 4;
  uint64_t* p_full = bars + 7;
  uint64_t* o_full = bars + 10;                // [2]: a unit's last P V done
  uint64_t* o_empty = bars + 12;               // [2]: O read by the epilogue
  uint64_t* stat_full = bars + 14;             // [2 parities][2 tiles]: a unit's row sums written
  uint64_t* k_full = bars + 18;                // [kStages] each
  uint64_t* k_empty = k_full + P::kStages;
  uint64_t* v_full = k_empty + P::kStages;
  uint64_t* v_ready = v_full + P::kStages;     // rows past the last key zeroed
  uint64_t* v_empty = v_ready + P::kStages;
  uint64_t* f_full = v_empty + P::kStages;      // [kFeedSlots] each: the ring of units
  uint64_t* f_empty = f_full + kFeedSlots;
  uint64_t* o_step = f_empty + kFeedSlots;     // a P V of a unit with one tile done
  uint64_t* done_bar = o_step + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(done_bar + 2);
  static_assert(18 + 5 * P::kStages + 2 * kFeedSlots + 4 <= 64, "barrier area holds 64 words");
  float2* stat = reinterpret_cast<float2*>(smem + P::kStat);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (!segments_ok(a, status)) {
    if (a.fill) refuse_rows(a.out, a.lse, a.N * a.H, DH / 8);
    return;
  }
  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], 1);
      mbar_init(&q_empty[x], 1);
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 128);
      mbar_init(&o_full[x], 1);
      mbar_init(&o_empty[x], 128);
      mbar_init(&stat_full[x], 128);
      mbar_init(&stat_full[2 + x], 128);
    }
    for (int s = 0; s < P::kStages; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_ready[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int s = 0; s < kFeedSlots; ++s) {
      mbar_init(&f_full[s], 1);
      mbar_init(&f_empty[s], kFeedReaders);
    }
    mbar_init(&s_full[2], 1);
    mbar_init(&p_full[2], 128);
    mbar_init(o_step, 1);
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // TMEM: S and P of tile A [0, 128), of tile B [128, 256), O of A [256, ..), O of B [384, ..)
  auto tS = [tmem](int x) { return tmem + (uint32_t)(x * 128); };
  auto tO = [tmem](int x) { return tmem + 256u + (uint32_t)(x * 128); };
  WaitCtx wc{abort_flag, status, wait_ns};
  const int share = a.H / a.Hkv;
  Feed feed{reinterpret_cast<int4*>(smem + P::kFeed), f_full, f_empty, 0};
  XUnit u{};

  if (warp < 4) {
    if (warp == 0 && lane == 0) {
      // -------------------------------------------------------------- K and V tiles
      if (a.L > 0) {
        tma_prefetch_desc(&m.k);
        tma_prefetch_desc(&m.v);
      }
      const uint64_t keep = l2_policy_evict_last();
      uint32_t t = 0;
      bool ok = true, kv_pending = false;  // kv_pending: the last K has no V behind it
      while (ok && feed.next<false>(u, wc)) {
        const int n = ((u.k1 - u.k0 + kTile - 1) / kTile);
        const int hk = xg.r > 1 ? u.g : u.g / share;
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
          const int s = (int)(t % P::kStages);
          const uint32_t ph = ((t / P::kStages) & 1) ^ 1;
          const int row = u.k0 + j * kTile;
          if (!wait_for(&k_empty[s], ph, wc)) { ok = false; break; }
          if (withhold && t == 0) { ok = false; break; }  // test hook: this tile never comes
          load_tile<DH>(&m.k, m.kv, &k_full[s], smem + P::kK + s * P::kTileBytes, 1, hk, row, keep);
          kv_pending = true;
          if (!wait_for(&v_empty[s], ph, wc)) { ok = false; break; }
          load_tile<DH>(&m.v, m.vv, &v_full[s], smem + P::kV + s * P::kTileBytes, 1, hk, row, keep);
          kv_pending = false;
          ++t;
        }
      }
      // Every load has landed before the CTA exits.
      volatile int zero = 0;
      WaitCtx dc{&zero, nullptr, 100000000ull};
      const uint32_t tk = t + (kv_pending ? 1 : 0);
      for (uint32_t s = 0; s < (uint32_t)P::kStages; ++s) {
        if (s < tk) wait_for(&k_full[s], ((tk - 1 - s) / P::kStages) & 1, dc);
        if (s < t) wait_for(&v_full[s], ((t - 1 - s) / P::kStages) & 1, dc);
      }
    } else if (warp == 3) {
      // -------------------------------------------------------------- units, and their query tiles
      if (lane == 0) tma_prefetch_desc(&m.q);
      const uint64_t once = l2_policy_evict_first();
      const WaitCtx wu = unit_wait(wc);
      uint32_t n0 = 0, n1 = 0;  // tiles A, B loaded
      Walk it(a, xg, 2 * xg.tokens, false);
      while (true) {
        int place;
        const bool more = it.next(u, place);
        u.q0 += place * 2 * xg.tokens;
        take_share(u.k0, u.k1, kTile, u.split, xg.splits);
        int go = 1;
        if (lane == 0) {
          go = feed.put(u, more ? 1 : 0, wu);
          if (go && more && u.k1 > u.k0) {
            const int head = u.g << xg.log2r;
            go = wait_for(&q_empty[0], (n0 & 1) ^ 1, wu);
            if (go) {
              load_tile<DH>(&m.q, m.qv, &q_full[0], smem + P::kQ, xg.r, head, u.q0, once);
              ++n0;
            }
            if (go && u.q0 + xg.tokens < u.q1) {
              go = wait_for(&q_empty[1], (n1 & 1) ^ 1, wu);
              if (go) {
                load_tile<DH>(&m.q, m.qv, &q_full[1], smem + P::kQ + P::kTileBytes, xg.r, head, u.q0 + xg.tokens, once);
                ++n1;
              }
            }
          }
        }
        if (!__shfl_sync(0xffffffffu, go, 0) || !more) break;
      }
      volatile int zero = 0;
      WaitCtx dc{&zero, nullptr, 100000000ull};
      if (lane == 0 && n0 > 0) wait_for(&q_full[0], (n0 - 1) & 1, dc);
      if (lane == 0 && n1 > 0) wait_for(&q_full[1], (n1 - 1) & 1, dc);
    } else if (warp == 2) {
      // -------------------------------------------------------------- rows past the last key
      uint32_t t = 0;
      bool ok = true;
      // Lane 0 reads the units and waits for the tiles.
      while (ok) {
        int w = 1;
        if (lane == 0) w = feed.next<false>(u, wc);
        if (!__shfl_sync(0xffffffffu, w, 0)) break;
        const int keys = __shfl_sync(0xffffffffu, u.k1 - u.k0, 0), n = (keys + kTile - 1) / kTile;
#pragma unroll 1
        for (int j = 0; j < n; ++j, ++t) {
          const int s = (int)(t % P::kStages);
          w = 1;
          if (lane == 0) w = wait_for(&v_full[s], (t / P::kStages) & 1, wc);
          if (!__shfl_sync(0xffffffffu, w, 0)) { ok = false; break; }
          __syncwarp();
          zero_rows<DH>(smem + P::kV + s * P::kTileBytes, keys - j * kTile, lane);
          if (lane == 0) mbar_arrive(&v_ready[s]);
        }
      }
    } else if (warp == 1) {
      // -------------------------------------------------------------- products
      // The whole warp walks the steps, one elected lane issues (a single
      // lane in the role took 12 % longer: nothing in it counts as uniform).
      // The loop over tiles is unrolled: as values they cost 8 %.
      const bool leader = elect_one();
      // 32-bit descriptor arithmetic (the high words are constant) keeps the issue short.
      constexpr uint32_t idS = idesc_bf16(128, 128, false, false);
      constexpr uint32_t idO = idesc_bf16(128, DH, false, true);
      const uint32_t q_lo = desc_lo(smem_u32(smem + P::kQ), 16), k_lo = desc_lo(smem_u32(smem + P::kK), 16),
                     v_lo = desc_lo(smem_u32(smem + P::kV), P::kChunk);
      uint32_t kt = 0, vt = 0;             // key and value tiles taken
      uint32_t qph = 0, pph = 0, oph = 0;  // phases of q_full, p_full, o_empty: bit x
      uint32_t used = 0;                   // bit x: tile x has had a unit
      XUnit nu{};                          // the next unit with keys
      bool left = true;                    // units may be left
      int n = 0, j = 0;
      bool have = false;                   // before the first unit there is no step, only the next S
      while (true) {
        const bool more = have && j + 1 < n;
        bool next = more;                  // is there an S to issue
        if (!more)
          while (left && !next) {
            left = feed.next<true>(nu, wc);
            next = left && nu.k1 > nu.k0;
          }
        if (!have && !next) break;
        const int valid = u.k1 - u.k0 - j * kTile;
        const int nvalid = more ? valid - kTile : nu.k1 - nu.k0;
        const bool nb = more ? u.q0 + xg.tokens < u.q1 : nu.q0 + xg.tokens < nu.q1;
        const int vs = (int)(vt % P::kStages), ks = (int)(kt % P::kStages);
        const uint32_t kph = (kt / P::kStages) & 1;
        if (have && !wait_for(&v_ready[vs], (vt / P::kStages) & 1, wc)) break;
        if (more && !wait_for(&k_full[ks], kph, wc)) break;
        int y = 0;                         // the next S to issue
        bool ok = true;
        const bool single = kOne && have && u.q0 + xg.tokens >= u.q1;
        if (kOne && single) {
          // One query tile: its S takes turns in the two buffers, S(j + 1)
          // before P V(j), so that a step is as long as the softmax.
          if (more) {
            tc_fence_after();
            if (leader) {
              const uint32_t kd = k_lo + (uint32_t)(ks * (P::kTileBytes >> 4)), ts = tS((j + 1) & 1);
#pragma unroll
              for (int kk = 0; kk < DH / 16; ++kk) {
                const uint32_t o = ((kk >> 2) * P::kChunk + (kk & 3) * 32) >> 4;
                umma_lo(ts, q_lo + o, kd + o, idS, (uint32_t)kk);
              }
              umma_commit(&s_full[(j & 1) ? 0 : 2]);
              if (nvalid <= kTile) umma_commit(&q_empty[0]);
            }
            y = 2;  // nothing is left to issue
          }
          const int b = (j & 1) ? 2 : 0;
          ok = wait_for(&p_full[b], (pph >> b) & 1, wc);
          pph ^= 1u << b;
          if (j == 0) {
            if (ok && (used & 1)) {
              ok = wait_for(&o_empty[0], oph & 1, wc);
              oph ^= 1u;
            }
            used |= 1u;
          }
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            const uint32_t vd = v_lo + (uint32_t)(vs * (P::kTileBytes >> 4)), ts = tS(j & 1);
            const int steps = min(valid + 15, kTile) >> 4;
#pragma unroll 4
            for (int kk = 0; kk < steps; ++kk) umma_ts_lo(tO(0), ts + kk * 8, vd + kk * 128, idO, (uint32_t)(j + kk));
            umma_commit(o_step);
            if (!more) umma_commit(&o_full[0]);
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (!ok) break;
          if (have && !single && (x == 0 || kOne || u.q0 + xg.tokens < u.q1)) {
            // O_x += P_x V in steps of 16 keys, once P is written and O_x free of the unit before
            ok = wait_for(&p_full[x], (pph >> x) & 1, wc);
            pph ^= 1u << x;
            if (j == 0) {
              if (ok && ((used >> x) & 1)) {
                ok = wait_for(&o_empty[x], (oph >> x) & 1, wc);
                oph ^= 1u << x;
              }
              used |= 1u << x;
            }
            if (!ok) break;
            tc_fence_after();
            uint32_t vd = v_lo + (uint32_t)(vs * (P::kTileBytes >> 4));
            uint32_t ts = tS(x);
            const uint32_t to = tO(x);
            if (!leader) {
            } else if (valid >= kTile) {
#pragma unroll
              for (int kk = 0; kk < kTile / 16; ++kk) umma_ts_lo(to, ts + kk * 8, vd + kk * 128, idO, (uint32_t)(j + kk));
            } else {
#pragma unroll 1
              for (int kk = 0; kk * 16 < valid; ++kk, ts += 8, vd += 128) umma_ts_lo(to, ts, vd, idO, (uint32_t)(j + kk));
            }
            if (!more && leader) umma_commit(&o_full[x]);
          }
          if (!next) continue;
          // At a unit's end S_A of the next one goes before this one's PV_B if its operands are here.
          if (x == 0 && !more && have && !single && !(mbar_test(&k_full[ks], kph) && mbar_test(&q_full[0], qph & 1))) continue;
#pragma unroll 1
          for (; y <= x && ok; ++y) {
            if (y == 1 && !nb) break;
            if (!more) {
              ok = (y == 1 || wait_for(&k_full[ks], kph, wc)) && wait_for(&q_full[y], (qph >> y) & 1, wc);
              qph ^= 1u << y;
              if (!ok) break;
            }
            tc_fence_after();
            // S_y = Q_y K^T over all 128 rows of the key tile: what lies past the last key is masked
            const uint32_t qd = q_lo + (uint32_t)(y * (P::kTileBytes >> 4)), kd = k_lo + (uint32_t)(ks * (P::kTileBytes >> 4));
            const uint32_t ts = tS(y);
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < DH / 16; ++kk) {
                const uint32_t o = ((kk >> 2) * P::kChunk + (kk & 3) * 32) >> 4;
                umma_lo(ts, qd + o, kd + o, idS, (uint32_t)kk);
              }
              umma_commit(&s_full[y]);
              if (nvalid <= kTile) umma_commit(&q_empty[y]);  // the unit's last S
            }
          }
        }
        if (!ok) break;
        if (have) {
          if (leader) umma_commit(&v_empty[vs]);
          ++vt;
        }
        if (next) {
          if (leader) umma_commit(&k_empty[ks]);
          ++kt;
        }
        if (more) {
          ++j;
        } else {
          u = nu;
          n = ((u.k1 - u.k0 + kTile - 1) / kTile);
          j = 0;
          have = next;
        }
      }
      if (leader) umma_commit(done_bar);
      volatile int zero = 0;
      WaitCtx dc{&zero, nullptr, 100000000ull};
      wait_for(done_bar, 0, dc);
    }
  } else if (warp < 12) {
    // ---------------------------------------------------------------- softmax
    const int x = (warp - 4) >> 2, sub = warp & 3, row = sub * 32 + lane;
    const uint32_t lane_base = (uint32_t)(sub * 32) << 16;
    const uint32_t tOx = tO(x) + lane_base;
    const float scale_log2 = 1.4426950408889634f * rsqrtf((float)DH);
    uint32_t sph = 0, un = 0;  // phases of s_full: bit by barrier
    uint32_t ones = 0;         // steps of units with one tile so far
    // Tile B's warps pass over units without one, and then wait for as long as
    // such a unit takes, for the next unit or for its first S.
    const WaitCtx wx = x ? unit_wait(wc) : wc;
    bool ok = true;
    while (ok && feed.next<true>(u, wx)) {
      const int n = (u.k1 - u.k0 + kTile - 1) / kTile;
      const bool alone = u.q0 + xg.tokens >= u.q1, single = kOne && alone;  // tile A takes turns in both buffers
      if (n == 0 || (alone && x == 1)) continue;
      float m_run = kNoMax;
      uint64_t l2 = f2_pack(0.f, 0.f);
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        const int odd = single ? j & 1 : 0;
        const int buf = odd ? 2 : x;
        const uint32_t tSx = tS(x + odd) + lane_base;
        if (!wait_for(&s_full[buf], (sph >> buf) & 1, wx)) { ok = false; break; }
        sph ^= 1u << buf;
        tc_fence_after();
        const int valid = u.k1 - u.k0 - j * kTile;
        if (valid < kTile) {
          // Columns past the last key: -inf, written to TMEM (as selects on
          // the registers they were a sixth of the kernel's instructions).
          const float inf = -INFINITY;
          int c = valid;
#pragma unroll 1
          for (; c & 15; ++c) tmem_st1(tSx + c, inf);
#pragma unroll 1
          for (; c < kTile; c += 16) {
            float v[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = inf;
            tmem_st16u(tSx + c, reinterpret_cast<const uint32_t*>(v));
          }
          tmem_st_wait();
        }
        // Half of the row at a time in registers, the first half last so that
        // it need not be read again: the exponentials below are then one loop
        // body of 64 columns.  Unrolled over all 128 the kernel's running code
        // did not fit the instruction cache (12 % of fetches missed).
        float sr[64];
        float mx = -INFINITY;
#pragma unroll 1
        for (int half = 1; half >= 0; --half) {
          tmem_ld32(tSx + half * 64, sr);
          tmem_ld32(tSx + half * 64 + 32, sr + 32);
          tmem_ld_wait();
          float m4[4];  // four chains of three-input maxima
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            m4[i] = fmax3(sr[16 * i], sr[16 * i + 1], sr[16 * i + 2]);
#pragma unroll
            for (int k = 3; k + 1 < 16; k += 2) m4[i] = fmax3(m4[i], sr[16 * i + k], sr[16 * i + k + 1]);
            m4[i] = fmaxf(m4[i], sr[16 * i + 15]);
          }
          mx = fmax3(mx, fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        }
        const float m_new = fmaxf(m_run, mx);
        // The maximum moves, and O is rescaled, only when the exponent would
        // pass 8; P and l share the older one otherwise.
        float alpha = 1.0f;
        bool rescale = false;
        if (j == 0) {
          m_run = m_new;
        } else {
          const bool need = (m_new - m_run) * scale_log2 > 8.0f;
          rescale = __any_sync(0xffffffffu, need);
          if (need) {
            alpha = P_moved(m_run, m_new, scale_log2);
            l2 = f2_mul(l2, f2_pack(alpha, alpha));
            m_run = m_new;
          }
        }
        // P = 2^(S scale - m scale) to bf16, the operand's type: rounding it by 2^-8
        // of itself at most is what O's own rounding may cost.  l sums it unrounded.
        uint64_t sc2, nm2;
        P_factors(m_run, scale_log2, sc2, nm2);
        uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll 1
        for (int half = 0; half * 64 < min(valid, kTile); ++half) {  // P V stops at the last key's 16
          if (half) {
            tmem_ld32(tSx + 64, sr);
            tmem_ld32(tSx + 96, sr + 32);
            tmem_ld_wait();
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float t0, t1;
              f2_unpack(f2_fma(f2_pack(sr[c * 32 + 2 * e], sr[c * 32 + 2 * e + 1]), sc2, nm2), t0, t1);
              t0 = fast_exp2(t0);
              t1 = fast_exp2(t1);
              acc[e & 3] = f2_add(acc[e & 3], f2_pack(t0, t1));
              pk[e] = pack_bf16x2(t0, t1);
            }
            tmem_st16u(tSx + half * 32 + c * 16, pk);
          }
        }
        l2 = f2_add(l2, f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])));
        if (single) {  // S(j) does not say that P V(j - 1) is done, as it does with two tiles
          if (ones > 0 && !wait_for(o_step, (ones - 1) & 1, wc)) { ok = false; break; }
          ++ones;
          tc_fence_after();
        }
        if (rescale) {
#pragma unroll 1
          for (int c = 0; c < DH; c += 16) {
            float o[16];
            tmem_ld16(tOx + c, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] *= alpha;
            tmem_st16u(tOx + c, reinterpret_cast<const uint32_t*>(o));
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_full[buf]);
      }
      if (!ok) break;
      float l0, l1;
      f2_unpack(l2, l0, l1);
      const float l = l0 + l1;
      // The slot of unit un + 2 is written only after the epilogue of unit un
      // has freed O, which P V of unit un + 1 waited for.
      stat[(un & 1) * 2 * kTile + x * kTile + row] = make_float2(l, m_run);
      mbar_arrive(&stat_full[(un & 1) * 2 + x]);
      ++un;
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const WaitCtx wu = unit_wait(wc);
    const int sub = warp & 3, row = sub * 32 + lane;
    const uint32_t lane_base = (uint32_t)(sub * 32) << 16;
    uint8_t* stage = smem + P::kStage + sub * 4096;
    uint32_t un0 = 0, un1 = 0;  // units of tile A, B
    bool ok = true;
    while (ok && feed.next<true, 100>(u, wu)) {
      const bool keys = u.k1 > u.k0;
#pragma unroll 1
      for (int x = 0; x < 2; ++x) {
        const int tok0 = u.q0 + x * xg.tokens;
        if (tok0 >= u.q1) break;
        float2 st = make_float2(0.0f, kNoMax);
        if (keys) {
          const uint32_t n = x ? un1++ : un0++;
          if (!wait_for<100>(&stat_full[(n & 1) * 2 + x], (n >> 1) & 1, wu) ||
              !wait_for<20>(&o_full[x], n & 1, wu)) { ok = false; break; }
          tc_fence_after();
          st = stat[(n & 1) * 2 * kTile + x * kTile + row];
        }
        // This thread's row: token and query head.
        auto place = [&](int r, int& tok, int& h) {
          tok = tok0 + (r >> xg.log2r);
          h = (u.g << xg.log2r) + (r & (xg.r - 1));
          return tok < u.q1;
        };
        int tok, h;
        const bool live = place(row, tok, h);
        if (part_o) {
          if (live) part_lm[((int64_t)u.split * a.H + h) * a.N + tok] = st;
        } else if (a.lse && live) {
          a.lse[(int64_t)h * a.N + tok] = lse_of(st.x, st.y, 1.4426950408889634f * rsqrtf((float)DH));
        }
        // l is at least 2^-16, or 0 where every score is -inf: as without keys
        st.x = st.x == 0.0f ? 0.0f : __fdividef(1.0f, st.x);
        if (part_o && !keys) continue;  // the join leaves a share without keys out
        const uint32_t to = tO(x) + lane_base;
        const int piece = lane & 7, sub8 = lane >> 3;
        uint8_t* mine = stage + lane * 128;
        // 128 bytes of each of the warp's rows go through shared memory at a
        // time: written by row, read back as whole 128-byte pieces, four rows
        // to a store.
        auto store_rows = [&](uint8_t* base, int row_bytes) {
          __syncwarp();
          uint4 v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + sub8;
            v[i] = *reinterpret_cast<const uint4*>(stage + r * 128 + ((piece ^ (r & 7)) << 4));
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            int t, hh;
            if (place(sub * 32 + i * 4 + sub8, t, hh))
              __stcs(reinterpret_cast<uint4*>(base + (int64_t)(t * a.H + hh) * row_bytes + piece * 16), v[i]);
          }
          __syncwarp();
        };
        if (!part_o) {
#pragma unroll 1
          for (int c = 0; c < DH / 64; ++c) {
            float o[64];
            tmem_ld32(to + c * 64, o);
            tmem_ld32(to + c * 64 + 32, o + 32);
            tmem_ld_wait();
            if (keys && c + 1 == DH / 64) {  // all of O is read
              tc_fence_before();
              mbar_arrive(&o_empty[x]);
            }
#pragma unroll
            for (int p = 0; p < 8; ++p) {
              uint4 w;
              w.x = pack_bf16x2(o[8 * p] * st.x, o[8 * p + 1] * st.x);
              w.y = pack_bf16x2(o[8 * p + 2] * st.x, o[8 * p + 3] * st.x);
              w.z = pack_bf16x2(o[8 * p + 4] * st.x, o[8 * p + 5] * st.x);
              w.w = pack_bf16x2(o[8 * p + 6] * st.x, o[8 * p + 7] * st.x);
              if (!keys) w = make_uint4(0, 0, 0, 0);  // what TMEM holds then is old
              *reinterpret_cast<uint4*>(mine + ((p ^ (lane & 7)) << 4)) = w;
            }
            store_rows(static_cast<uint8_t*>(a.out) + c * 128, DH * 2);
          }
        } else {  // a share of the keys: O / l in fp32
          uint8_t* base = reinterpret_cast<uint8_t*>(part_o + (int64_t)u.split * a.N * a.H * DH);
#pragma unroll 1
          for (int c = 0; c < DH / 32; ++c) {
            float o[32];
            tmem_ld32(to + c * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int p = 0; p < 8; ++p)
              *reinterpret_cast<float4*>(mine + ((p ^ (lane & 7)) << 4)) =
                  make_float4(o[4 * p] * st.x, o[4 * p + 1] * st.x, o[4 * p + 2] * st.x, o[4 * p + 3] * st.x);
            if (c + 1 == DH / 32) {
              tc_fence_before();
              mbar_arrive(&o_empty[x]);
            }
            store_rows(base + c * 128, DH * 4);
          }
        }
      }
    }
    fill_rows<DH>(a, a.out, a.lse, (int64_t)blockIdx.x * 128 + threadIdx.x - 384, (int64_t)gridDim.x * 128);
    if (xg.splits == 1) empty_segments<DH>(a, a.out, a.lse, blockIdx.x * 4 + warp - 12, gridDim.x * 4);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// out and lse from the shares' O_s = O / l and (l_s, m_s): with m the largest m_s
// and w_s = l_s 2^((m_s - m) scale), out = sum_s w_s O_s / sum_s w_s.  One warp
// per (token, head) of a segment; a share without keys has l = 0.  Two numbers
// and not lse alone, which loses l where m is large.
template <int DH>
__global__ void __launch_bounds__(256) cross_join_kernel(const CrossArgs a, int splits, const float* __restrict__ part_o,
                                                         const float2* __restrict__ part_lm, int* status) {
  constexpr int C = DH / 32;
  if (!segments_ok(a, nullptr)) return;  // the kernel before reported it
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (w >= a.N * a.H) return;
  const int64_t n = w / a.H;
  const int h = (int)(w - n * a.H);
  bool inside = a.q_off == nullptr;
  if (!inside) inside = n >= a.q_off[0] && n < a.q_off[a.S];  // segments follow one another
  if (!inside) return;
  const int64_t rows = a.N * a.H, at = (int64_t)h * a.N + n;
  const float scale_log2 = 1.4426950408889634f * rsqrtf((float)DH);
  float m = kNoMax;
  for (int s = lane; s < splits; s += 32) m = fmaxf(m, part_lm[s * rows + at].y);
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
  float l = 0.0f, o[C] = {};
  const float* p = part_o + w * DH + lane * C;
  for (int base = 0; base < splits; base += 32) {
    // 32 weights at a time, one a lane; the rows of the shares with keys
    // then come in several at once
    const float2 e = base + lane < splits ? part_lm[(base + lane) * rows + at] : make_float2(0.0f, m);
    const float f = e.x * P_moved(e.y, m, scale_log2);
#pragma unroll 8
    for (int s = 0; s < min(32, splits - base); ++s) {
      const float g = __shfl_sync(0xffffffffu, f, s);
      l += g;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const float v = g > 0.0f ? p[(base + s) * rows * DH + i] : 0.0f;
        o[i] = fmaf(g, v, o[i]);
      }
    }
  }
  store_row<C>(a.out, w * DH, lane, o, l == 0.0f ? 0.0f : 1.0f / l);
  if (a.lse && lane == 0) a.lse[at] = lse_of(l, m, scale_log2);
}


// Shares of the keys: enough units for every SM, each of two key tiles at least.
int splits_of(int64_t N, int64_t L, int H, int r, int S) {
  return shares(places_most(N, 2 * kTile / r, S) * (H / r), ceil_div(L, S), kTile, kSplitSms);
}

template <int DH>
cudaError_t launch_fwd(const DevCtx& c, const CrossArgs& a, uint8_t* ws, int* launches) {
  using P = XPlan<DH>;
  XMaps m{};
  XGrid x = pack_grid(pack_of(a));
  x.heads = a.H / x.r;
  x.splits = splits_of(a.N, a.L, a.H, x.r, a.S);
  bool ok = view_2d(&m.k, &m.kv, a.k, a.k_sn, a.k_sh, a.L, a.Hkv, DH) &&
            view_2d(&m.v, &m.vv, a.v, a.v_sn, a.v_sh, a.L, a.Hkv, DH);
  ok = ok && (x.r > 1 ? make_tmap_heads(&m.q, a.q, DH, a.H, a.N, a.q_sh, a.q_sn, x.r, x.tokens)
                      : view_2d(&m.q, &m.qv, a.q, a.q_sn, a.q_sh, a.N, a.H, DH));
  if (!ok) return cudaErrorInvalidValue;
  float* po = nullptr;
  float2* pl = nullptr;
  if (x.splits > 1) {
    pl = reinterpret_cast<float2*>(ws);
    po = reinterpret_cast<float*>(ws + align_up((size_t)x.splits * a.N * a.H * 8, 256));
  }
  const bool one = a.N <= (int64_t)a.S * x.tokens;
  const auto kernel = one ? cross_fwd_kernel<DH, true> : cross_fwd_kernel<DH, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, P::kBytes);
  if (e != cudaSuccess) return e;
  const int64_t units = places_most(a.N, 2 * x.tokens, a.S) * x.splits * x.heads;
  const unsigned grid = (unsigned)std::min<int64_t>(units, c.num_sms);
  set_steps(&x, grid);
  kernel<<<grid, kXThreads, P::kBytes, c.stream>>>(m, a, x, po, pl, a.withhold, c.status, (unsigned long long)c.wait_ns);
  *launches = 1;
  if ((e = cudaGetLastError()) != cudaSuccess || x.splits == 1) return e;
  cross_join_kernel<DH><<<(unsigned)ceil_div(a.N * a.H, 8), 256, 0, c.stream>>>(a, x.splits, po, pl, c.status);
  *launches = 2;
  return cudaGetLastError();
}

}  // namespace

size_t cross_fwd_ws_bytes(int64_t N, int64_t L, int H, int H_kv, int d_h, int S) {
  // Packed or not is known with the strides only: the larger of the two.
  size_t most = 0;
  for (int r : {1, H / H_kv}) {
    if (r < 1 || r > 64 || (r & (r - 1))) continue;
    const int64_t splits = splits_of(N, L, H, r, S);
    if (splits > 1) most = std::max(most, align_up((size_t)(splits * N * H * 8), 256) + (size_t)(splits * N * H * d_h * 4));
  }
  return most;
}

cudaError_t launch_cross_attn(const DevCtx& c, const CrossArgs& a, uint8_t* ws, int* launches) {
  *launches = 0;
  if (a.N == 0) return cudaSuccess;
  return a.d_h == 128 ? launch_fwd<128>(c, a, ws, launches) : launch_fwd<64>(c, a, ws, launches);
}

}  // namespace moga

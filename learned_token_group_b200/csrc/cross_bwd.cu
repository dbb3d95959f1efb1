// Gradients of cross attention (the forward and its conventions are in
// cross.cu).  With P = exp(S - lse), dP = dO V^T, D = rowsum(dO * O) and
// dS = P * (dP - D):
//   dQ = dS K / sqrt(d_h),   dK = dS^T Q / sqrt(d_h),   dV = P^T dO.
//
// Two passes, each with S and dP anew: 14 instead of 10 flops per pair and
// channel.  One pass would have to add every key tile's share of dQ, 64 KB of
// fp32 for a tile of each kind, outside the SM: more bytes than the products
// saved, in an order that changes.
//
// cross_dq_kernel   a unit is one 128-row query tile (rows as in the forward:
//   128 / r tokens of r heads) and its segment's keys.  Per key tile t:
//   dP(t), dQ(t - 1), S(t + 1), across units, so that a prompt of a few tiles
//   leaves no gap between one unit and the next.
// cross_dkv_kernel  a unit is one 128-row key tile of a key head and a share of
//   its segment's queries, over the query heads that share the key head.  Per
//   query tile t: S^T(t), dV and dK (t - 1), dP^T(t).  Prompts have few key
//   tiles (512 keys of 12 heads: 48 for 148 SMs), so the queries are split and
//   the shares' fp32 sums added by cross_sum_kernel in a fixed order.
//
// Warp 0 loads K and V (dQ) or Q and dO (dK, dV), warp 3 the stationary tiles
// of the units it walks, warp 1 issues the products, warp 2 zeroes rows past
// a segment's end (and brings lse and D of the query rows), warps 4-11 turn S
// and dP into bf16 P and dS (two warpgroups, 64 columns each) in the TMEM
// columns that S had, which the closing products read as their A operand;
// warps 12-15 write the results and, for dQ, compute D a unit ahead.
//
// Measured at 187,200 x 512 keys, 12 heads of 128 channels: dQ 0.94 ms (0.94
// PFLOP/s over its three products; a key tile takes 2,900 cycles, most of them
// the softmax warps'), dK and dV 0.94 ms (1.25 PFLOP/s over four; 3,020 cycles
// a tile, tensor pipe 68 % active: the next S^T waits until dP^T is read).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "cross.cuh"

namespace moga {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

struct BMaps {
  CUtensorMap q, dout, out, k, v;
  XView qv, dv, kv, vv;  // out is laid out as dout
};

template <int DH>
struct BPlan {
  static constexpr int T = kTile * DH * 2;        // bytes of a tile
  static constexpr int kChunk = kTile * 128;
  // dQ: Q, dO, K ring of three, V ring of two.  K is read by S and, a tile
  // later, by dQ; V by dP alone.  S of a unit's last tile is issued a tile
  // ahead, so the next unit's Q has a tile's time to come.
  static constexpr int kQ = 0, kDO = T, kK = 2 * T, kV = 5 * T;
  // dK, dV: K, V, query ring of three, dO ring of two.
  static constexpr int kX1 = 0, kX2 = T, kY1 = 2 * T, kY2 = 5 * T;
  static constexpr int kVec = 7 * T;              // fp32 vectors (dQ: 2 KB; dK, dV: 2.5 KB)
  static constexpr int kFeed = kVec + 5 * kTile * 4;
  static constexpr int kBar = kFeed + kFeedSlots * 32;
  static constexpr int kBytes = kBar + 384;
  static_assert(kBytes <= 232448, "shared memory");
};

// The dynamic shared memory of a kernel without static shared memory starts
// on a 1 KB boundary; the tiles need it and there is no room to move them.
__device__ __forceinline__ bool base_ok(const uint8_t* smem, int* status) {
  if ((smem_u32(smem) & 1023u) == 0) return true;
  if (threadIdx.x == 0 && status) atomicOr(status, DEV_RANGE);
  return false;
}

// A tile's 128 x 128 product of two K-major operands into TMEM.
template <int DH>
__device__ __forceinline__ void issue_nt(uint32_t d, uint32_t a_lo, uint32_t b_lo) {
  constexpr uint32_t id = idesc_bf16(128, 128, false, false);
#pragma unroll
  for (int kk = 0; kk < DH / 16; ++kk) {
    const uint32_t o = ((kk >> 2) * kTile * 128 + (kk & 3) * 32) >> 4;
    umma_lo(d, a_lo + o, b_lo + o, id, (uint32_t)kk);
  }
}
// d += A B over `valid` rows of B in steps of 16: A in TMEM, where warpgroup w
// wrote rows [64 w, 64 w + 64) of B as 32 columns from 64 w; B MN-major.
template <int DH>
__device__ __forceinline__ void issue_acc(uint32_t d, uint32_t a_tmem, uint32_t b_lo, int valid, bool acc) {
  constexpr uint32_t id = idesc_bf16(128, DH, false, true);
  if (valid >= kTile) {
#pragma unroll
    for (int kk = 0; kk < kTile / 16; ++kk)
      umma_ts_lo(d, a_tmem + 64 * (kk >> 2) + 8 * (kk & 3), b_lo + kk * 128, id, (acc || kk > 0) ? 1u : 0u);
  } else {
#pragma unroll 1
    for (int kk = 0; kk * 16 < valid; ++kk)
      umma_ts_lo(d, a_tmem + 64 * (kk >> 2) + 8 * (kk & 3), b_lo + kk * 128, id, (acc || kk > 0) ? 1u : 0u);
  }
}

// A whole 32-byte sector: each thread writes its own row, so that a store of
// 16 bytes would touch every sector twice.
__device__ __forceinline__ void store32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

__device__ __forceinline__ void load32(uint32_t* w, const void* p) {
  asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}

// One row of DH accumulators, scaled: bf16 to `out`, or fp32 to `part`.
template <int DH>
__device__ __forceinline__ void write_row(uint32_t taddr, float f, bool keep, bool live, __nv_bfloat16* out,
                                          float* part) {
#pragma unroll 1
  for (int c = 0; c < DH; c += 32) {
    float o[32];
    __syncwarp();
    tmem_ld32(taddr + c, o);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = keep ? o[e] * f : 0.0f;
    if (live && part) {
#pragma unroll
      for (int e = 0; e < 32; e += 8) store32(part + c + e, reinterpret_cast<const uint32_t*>(o + e));
    } else if (live) {
#pragma unroll
      for (int e = 0; e < 32; e += 16) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(o[e + 2 * i], o[e + 2 * i + 1]);
        store32(out + c + e, w);
      }
    }
  }
}

// p[0], p[1] = 2^(p scale + nl), in place.
__device__ __forceinline__ void exp2_pair(float* p, uint64_t sc2, uint64_t nl2) {
  float x, y;
  f2_unpack(f2_fma(f2_pack(p[0], p[1]), sc2, nl2), x, y);
  p[0] = fast_exp2(x);
  p[1] = fast_exp2(y);
}
// P (dP - D) of two columns, in bf16.
__device__ __forceinline__ uint32_t ds_pair(const float* p, const float* d, uint64_t md2) {
  float x, y;
  f2_unpack(f2_mul(f2_pack(p[0], p[1]), f2_add(f2_pack(d[0], d[1]), md2)), x, y);
  return pack_bf16x2(x, y);
}

// ------------------------------------------------------------------ dQ
template <int DH>
__global__ void __launch_bounds__(kXThreads, 1)
cross_dq_kernel(const __grid_constant__ BMaps m, const CrossArgs a, const XGrid xg, float* part, int* status,
                unsigned long long wait_ns) {
  using P = BPlan<DH>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (!base_ok(smem, status) || !segments_ok(a, status)) {
    if (a.fill) refuse_rows(a.dq, nullptr, a.N * a.H, DH / 8);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + P::kBar);
  uint64_t* q_full = bars;
  uint64_t* q_empty = bars + 1;
  uint64_t* do_full = bars + 2;
  uint64_t* do_empty = bars + 3;
  uint64_t* k_full = bars + 6;        // [3]
  uint64_t* k_ready = bars + 9;       // [3]: rows past the last key zeroed
  uint64_t* k_empty = bars + 12;      // [3]
  uint64_t* v_full = bars + 15;       // [2]
  uint64_t* v_ready = bars + 4;       // [2]
  uint64_t* v_empty = bars + 17;      // [2]
  uint64_t* s_full = bars + 19;       // [2]: S of tile t on t % 2
  uint64_t* d_full = bars + 38;       // dP computed
  uint64_t* dp_free = bars + 21;      // dP read
  uint64_t* p_full = bars + 22;       // [2]: dS of tile t written
  uint64_t* acc_full = bars + 24;
  uint64_t* acc_empty = bars + 25;
  uint64_t* vec_full = bars + 26;     // [2]: lse and D of a unit's rows
  uint64_t* f_full = bars + 28;       // [4]
  uint64_t* f_empty = bars + 32;      // [4]
  uint64_t* sum_bar = bars + 36;      // a row's two halves of D added
  uint64_t* done_bar = bars + 37;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 39);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 40);
  float* vec = reinterpret_cast<float*>(smem + P::kVec);  // [2 units][-lse log2 e, D][128]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 39; ++i) {
      const bool all = i == 21 || i == 22 || i == 23 || i == 36, epi = i == 25 || i == 26 || i == 27, feed = i >= 32 && i < 36;
      mbar_init(&bars[i], all ? 256 : epi ? 128 : feed ? kFeedReaders : 1);
    }
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
  // TMEM: S (then dS over it) of tile t at 0 or 384, dP at 128, dQ at 256
  auto tS = [tmem](uint32_t t) { return tmem + ((t & 1u) ? 384u : 0u); };
  const uint32_t tD = tmem + 128u, tQ = tmem + 256u;
  WaitCtx wc{abort_flag, status, wait_ns};
  Feed feed{reinterpret_cast<int4*>(smem + P::kFeed), f_full, f_empty, 0};
  XUnit u{};
  const int share = a.H / a.Hkv;
  volatile int zero = 0;
  WaitCtx dc{&zero, nullptr, 100000000ull};  // for loads and products in flight at the end

  if (warp == 0) {
    if (lane == 0) {
      // -------------------------------------------------------------- K and V
      const uint64_t keep = l2_policy_evict_last();
      uint32_t kt = 0, vt = 0;
      bool ok = true;
      while (ok && feed.next<false>(u, wc)) {
        const int hk = xg.r > 1 ? u.g : u.g / share;
#pragma unroll 1
        for (int row = u.k0; row < u.k1; row += kTile) {
          const uint32_t s = kt % 3, sv = vt % 2;
          if (!wait_for(&k_empty[s], ((kt / 3) & 1) ^ 1, wc)) { ok = false; break; }
          if (a.withhold && kt == 0) { ok = false; break; }  // test hook: this tile never comes
          load_tile<DH>(&m.k, m.kv, &k_full[s], smem + P::kK + s * P::T, 1, hk, row, keep);
          ++kt;
          if (!wait_for(&v_empty[sv], ((vt / 2) & 1) ^ 1, wc)) { ok = false; break; }
          load_tile<DH>(&m.v, m.vv, &v_full[sv], smem + P::kV + sv * P::T, 1, hk, row, keep);
          ++vt;
        }
      }
      for (uint32_t s = 0; s < 3; ++s)
        if (s < kt) wait_for(&k_full[s], ((kt - 1 - s) / 3) & 1, dc);
      for (uint32_t s = 0; s < 2; ++s)
        if (s < vt) wait_for(&v_full[s], ((vt - 1 - s) / 2) & 1, dc);
    }
  } else if (warp == 3) {
    // ---------------------------------------------------------------- units, their Q and dO tiles
    const WaitCtx wu = unit_wait(wc);
    const uint64_t once = l2_policy_evict_first();
    uint32_t n = 0, nd = 0;
    Walk it(a, xg, xg.tokens, false);
    while (true) {
      int place;
      const bool more = it.next(u, place);
      u.q0 += place * xg.tokens;
      const bool whole = u.k1 - u.k0 <= kTile;  // the unit's one tile holds its segment's keys
      take_share(u.k0, u.k1, kTile, u.split, xg.splits);
      int go = 1;
      if (lane == 0) {
        // bit 1 of the entry's flag: D comes from P and dP (see below)
        const int flag = more ? (whole && xg.splits == 1 ? 3 : 1) : 0;
        const int head = u.g << xg.log2r;
        if (flag == 1 && u.k1 > u.k0) {  // what D is computed from, a unit ahead
          prefetch_tile<DH>(&m.out, m.dv, xg.r, head, u.q0);
          prefetch_tile<DH>(&m.dout, m.dv, xg.r, head, u.q0);
        }
        go = feed.put(u, flag, wu);
        if (go && more && u.k1 > u.k0) {
          go = wait_for(q_empty, (n & 1) ^ 1, wu);
          if (go) {
            load_tile<DH>(&m.q, m.qv, q_full, smem + P::kQ, xg.r, head, u.q0, once);
            ++n;
            go = wait_for(do_empty, (nd & 1) ^ 1, wu);
          }
          if (go) {
            load_tile<DH>(&m.dout, m.dv, do_full, smem + P::kDO, xg.r, head, u.q0, once);
            ++nd;
          }
        }
      }
      if (!__shfl_sync(0xffffffffu, go, 0) || !more) break;
    }
    if (lane == 0) {
      if (n > 0) wait_for(q_full, (n - 1) & 1, dc);
      if (nd > 0) wait_for(do_full, (nd - 1) & 1, dc);
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------------- rows past the last key
    uint32_t t = 0;
    bool ok = true;
    while (ok) {
      int w = 1;
      if (lane == 0) w = feed.next<false>(u, wc);
      if (!__shfl_sync(0xffffffffu, w, 0)) break;
      const int keys = __shfl_sync(0xffffffffu, u.k1 - u.k0, 0);
#pragma unroll 1
      for (int j = 0; j * kTile < keys; ++j, ++t) {
        const uint32_t s = t % 3;
        if (lane == 0) w = wait_for(&k_full[s], (t / 3) & 1, wc);
        if (!__shfl_sync(0xffffffffu, w, 0)) { ok = false; break; }
        __syncwarp();
        zero_rows<DH>(smem + P::kK + s * P::T, keys - j * kTile, lane);
        if (lane == 0) {
          mbar_arrive(&k_ready[s]);
          w = wait_for(&v_full[t % 2], (t / 2) & 1, wc);
        }
        if (!__shfl_sync(0xffffffffu, w, 0)) { ok = false; break; }
        __syncwarp();
        zero_rows<DH>(smem + P::kV + (t % 2) * P::T, keys - j * kTile, lane);
        if (lane == 0) mbar_arrive(&v_ready[t % 2]);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- products
    const bool leader = elect_one();
    const uint32_t q_lo = desc_lo(smem_u32(smem + P::kQ), 16), do_lo = desc_lo(smem_u32(smem + P::kDO), 16),
                   k_lo = desc_lo(smem_u32(smem + P::kK), 16), kt_lo = desc_lo(smem_u32(smem + P::kK), P::kChunk),
                   v_lo = desc_lo(smem_u32(smem + P::kV), 16);
    XUnit nu{};
    bool left = true, have = false;      // units may be left; there is a unit
    int n = 0, j = 0;                    // its tiles, and this one
    uint32_t t = 0, un = 0;              // tiles and units so far (this one not)
    int wait_valid = 0;                  // keys of tile t - 1, whose dQ is open (0: none)
    bool wait_first = false, wait_last = false;
    uint32_t accs = 0;                   // units whose dQ has begun
    while (true) {
      bool ok = true;
      const bool more = have && j + 1 < n;
      if (have) {
        // dP(t)
        ok = wait_for(&v_ready[t % 2], (t / 2) & 1, wc) && (j > 0 || wait_for(do_full, un & 1, wc)) &&
             (t == 0 || wait_for(dp_free, (t - 1) & 1, wc));
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          issue_nt<DH>(tD, do_lo, v_lo + (t % 2) * (P::T >> 4));
          umma_commit(d_full);
          umma_commit(&v_empty[t % 2]);
          if (!more) umma_commit(do_empty);
        }
      }
      if (wait_valid > 0) {
        // dQ(t - 1)
        const uint32_t tp = t - 1;
        ok = wait_for(&p_full[tp & 1], (tp >> 1) & 1, wc);
        if (ok && wait_first) {
          if (accs > 0) ok = wait_for(acc_empty, (accs - 1) & 1, wc);
          ++accs;
        }
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          issue_acc<DH>(tQ, tS(tp), kt_lo + (tp % 3) * (P::T >> 4), wait_valid, !wait_first);
          umma_commit(&k_empty[tp % 3]);
          if (wait_last) umma_commit(acc_full);
        }
        wait_valid = 0;
      }
      // S of the next tile
      bool next = more;
      if (!more)
        while (left && !next) {
          left = feed.next<true>(nu, wc);
          next = left && nu.k1 > nu.k0;
        }
      const uint32_t t1 = have ? t + 1 : 0, un1 = more ? un : have ? un + 1 : 0;
      if (next) {
        ok = wait_for(&k_ready[t1 % 3], (t1 / 3) & 1, wc) && (more || wait_for(q_full, un1 & 1, wc));
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          issue_nt<DH>(tS(t1), q_lo, k_lo + (t1 % 3) * (P::T >> 4));
          umma_commit(&s_full[t1 & 1]);
          if (more ? j + 2 == n : nu.k1 - nu.k0 <= kTile) umma_commit(q_empty);  // the unit's last S
        }
      }
      if (!have && !next) break;
      if (have) {
        wait_valid = min(u.k1 - u.k0 - j * kTile, kTile);
        wait_first = j == 0;
        wait_last = !more;
      }
      if (more) {
        ++j;
      } else {
        u = nu;
        n = (u.k1 - u.k0 + kTile - 1) / kTile;
        j = 0;
        have = next;
      }
      t = t1;
      un = un1;
    }
    if (leader) umma_commit(done_bar);
    wait_for(done_bar, 0, dc);
  } else if (warp < 12) {
    // ---------------------------------------------------------------- dS
    const int wg = (warp - 4) >> 2, sub = warp & 3, row = sub * 32 + lane;
    const uint32_t at = ((uint32_t)(sub * 32) << 16) + 64 * wg;  // this warp's lanes, its warpgroup's columns
    const float scale_log2 = kLog2e * rsqrtf((float)DH);
    uint32_t t = 0, un = 0, sums = 0;
    bool ok = true;
    int flag;
    while (ok && (flag = feed.next_flag<true>(u, wc)) != 0) {
      if (u.k1 <= u.k0) continue;
      float* mine = vec + (un & 1) * 2 * kTile + row;
      if (!wait_for(&vec_full[un & 1], (un >> 1) & 1, wc)) break;
      const float nl = mine[0];
      float D = mine[kTile];
#pragma unroll 1
      for (int k = u.k0; k < u.k1; k += kTile, ++t) {
        if (!wait_for(&s_full[t & 1], (t >> 1) & 1, wc)) { ok = false; break; }
        tc_fence_after();
        const uint32_t ts = tS(t) + at;
        const uint64_t sc2 = f2_pack(scale_log2, scale_log2), nl2 = f2_pack(nl, nl);
        // 32 columns at a time, in one loop body: unrolled over both halves
        // the code that runs did not fit the instruction cache.
        auto load_p = [&](int c, float* p) {
          tmem_ld32(ts + c, p);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; e += 2) exp2_pair(p + e, sc2, nl2);
          const int valid = u.k1 - k - 64 * wg - c;
          if (valid < 32) {
#pragma unroll
            for (int e = 0; e < 32; ++e) p[e] = e < valid ? p[e] : 0.0f;
          }
        };
        if (flag & 2) {
          // One tile holds all of the row's keys: D = sum_j P_ij dP_ij, in
          // fp32.  From O, which is rounded to bf16, it would be the largest
          // error of the gradients where few keys make O as large as V.
          if (!wait_for(d_full, t & 1, wc)) { ok = false; break; }
          tc_fence_after();
          float sum = 0.0f;
#pragma unroll 1
          for (int c = 0; c < 64; c += 32) {
            float p[32], d[32];
            load_p(c, p);
            tmem_ld32(tD + at + c, d);
            tmem_ld_wait();
            const int valid = u.k1 - k - 64 * wg - c;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e < valid) sum = fmaf(p[e], d[e], sum);
          }
          atomicAdd(mine + kTile, sum);  // 0 and two terms: the same in either order
          mbar_arrive(sum_bar);
          ok = wait_for(sum_bar, sums & 1, wc);
          if (!ok) break;
          ++sums;
          D = mine[kTile];
          const int tok = u.q0 + (row >> xg.log2r);
          if (wg == 0 && tok < u.q1)
            a.dsum[(int64_t)((u.g << xg.log2r) + (row & (xg.r - 1))) * a.N + tok] = D;
        }
        const uint64_t md2 = f2_pack(-D, -D);
#pragma unroll 1
        for (int c = 0; c < 64; c += 32) {
          float p[32], d[32];
          load_p(c, p);
          if (c == 0 && !(flag & 2)) {
            ok = wait_for(d_full, t & 1, wc);
            if (!ok) break;
            tc_fence_after();
          }
          tmem_ld32(tD + at + c, d);
          tmem_ld_wait();
          if (c > 0) {
            tc_fence_before();
            mbar_arrive(dp_free);
          }
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) pk[e] = ds_pair(p + 2 * e, d + 2 * e, md2);
          tmem_st16u(ts + c / 2, pk);
        }
        if (!ok) break;
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_full[t & 1]);
      }
      ++un;
    }
  } else {
    // ---------------------------------------------------------------- D a unit ahead, and the results
    const WaitCtx wu = unit_wait(wc);
    const int sub = warp & 3, row = sub * 32 + lane;
    const uint32_t lanes = (uint32_t)(sub * 32) << 16;
    uint32_t un = 0, on = 0;
    XUnit pu{};
    bool pending = false, ok = true;
    auto write = [&](const XUnit& w, bool keys) {
      const int tok = w.q0 + (row >> xg.log2r), h = (w.g << xg.log2r) + (row & (xg.r - 1));
      const bool live = tok < w.q1;
      const int64_t o = live ? ((int64_t)tok * a.H + h) * DH : 0;
      write_row<DH>(tQ + lanes, rsqrtf((float)DH), keys, live, static_cast<__nv_bfloat16*>(a.dq) + o,
                    part ? part + (int64_t)w.split * a.N * a.H * DH + o : nullptr);
    };
    auto finish = [&]() {  // the unit before
      if (!wait_for<100>(acc_full, on & 1, wu)) return false;
      ++on;
      tc_fence_after();
      write(pu, true);
      tc_fence_before();
      mbar_arrive(acc_empty);
      return true;
    };
    int flag;
    while (ok && (flag = feed.next_flag<true, 100>(u, wu)) != 0) {
      const bool keys = u.k1 > u.k0;
      if (keys) {
        float* out = vec + (un & 1) * 2 * kTile;
        const int tok = u.q0 + (row >> xg.log2r), h = (u.g << xg.log2r) + (row & (xg.r - 1));
        const bool live = tok < u.q1;
        const float lse = live ? a.lse[(int64_t)h * a.N + tok] : INFINITY;
        float D = 0.0f;
        if (live && !(flag & 2)) {
          // A thread sums its own row, in whole sectors: rows shared by lanes
          // took more code, which this warp alone runs, once a unit.
          const int64_t o = ((int64_t)tok * a.H + h) * DH;
          const __nv_bfloat16 *px = static_cast<const __nv_bfloat16*>(a.dout) + o,
                              *py = static_cast<const __nv_bfloat16*>(a.out) + o;
#pragma unroll 1
          for (int c = 0; c < DH; c += 32) {
            uint32_t x[16], y[16];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              load32(x + 8 * i, px + c + 16 * i);
              load32(y + 8 * i, py + c + 16 * i);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              D = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), D);
              D = fmaf(__uint_as_float(x[i] & 0xffff0000u), __uint_as_float(y[i] & 0xffff0000u), D);
            }
          }
          if (u.split == 0) a.dsum[(int64_t)h * a.N + tok] = D;
        }
        out[row] = neg_lse_log2(lse);
        out[kTile + row] = D;
        mbar_arrive(&vec_full[un & 1]);
        ++un;
      }
      if (pending) ok = finish();
      pending = keys;
      if (keys) pu = u; else write(u, false);
    }
    if (ok && pending) finish();
    fill_rows<DH>(a, a.dq, nullptr, (int64_t)blockIdx.x * 128 + threadIdx.x - 384, (int64_t)gridDim.x * 128);
    if (xg.splits == 1) empty_segments<DH>(a, a.dq, nullptr, blockIdx.x * 4 + warp - 12, gridDim.x * 4);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ dK, dV
template <int DH>
__global__ void __launch_bounds__(kXThreads, 1)
cross_dkv_kernel(const __grid_constant__ BMaps m, const CrossArgs a, const XGrid xg, float* part, int* status,
                 unsigned long long wait_ns) {
  using P = BPlan<DH>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (!base_ok(smem, status) || !segments_ok(a, status)) return;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + P::kBar);
  uint64_t* x_full = bars;
  uint64_t* x_empty = bars + 1;
  uint64_t* y1_full = bars + 2;       // [3]: Q
  uint64_t* y1_ready = bars + 5;      // [3]: rows past the last query zeroed, lse there
  uint64_t* y1_empty = bars + 8;      // [3]
  uint64_t* y2_full = bars + 11;      // [2]: dO
  uint64_t* y2_ready = bars + 13;     // [2]: likewise, with D
  uint64_t* y2_empty = bars + 15;     // [2]
  uint64_t* s_full = bars + 17;
  uint64_t* d_full = bars + 18;
  uint64_t* dp_free = bars + 19;
  uint64_t* p_full = bars + 20;       // [2]
  uint64_t* acc_full = bars + 22;
  uint64_t* acc_empty = bars + 23;
  uint64_t* f_full = bars + 24;       // [4]
  uint64_t* f_empty = bars + 28;      // [4]
  uint64_t* done_bar = bars + 32;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 33);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 34);
  float* vec1 = reinterpret_cast<float*>(smem + P::kVec);  // [3][128]: -lse log2 e
  float* vec2 = vec1 + 3 * kTile;                          // [2][128]: -D
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 33; ++i) {
      const bool all = i == 19 || i == 20 || i == 21, feed = i >= 28 && i < 32;
      mbar_init(&bars[i], all ? 256 : i == 23 ? 128 : feed ? kFeedReaders : 1);
    }
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
  // TMEM: S^T of tile t (then P, and dS 32 columns on) in buffer t % 2 of two,
  // dP^T in the other; dV at 256, dK behind it.
  auto tS = [tmem](uint32_t t) { return tmem + 128u * (t & 1u); };
  auto tD = [tmem](uint32_t t) { return tmem + 128u * ((t & 1u) ^ 1u); };
  const uint32_t tV = tmem + 256u, tK = tmem + 256u + (uint32_t)DH;
  WaitCtx wc{abort_flag, status, wait_ns};
  Feed feed{reinterpret_cast<int4*>(smem + P::kFeed), f_full, f_empty, 0};
  XUnit u{};
  // A unit's query tiles: [q0, q1) in steps of xg.tokens, once, or (without
  // packing) once for every query head that shares the key head.
  const int loops = xg.r > 1 ? 1 : a.H / a.Hkv;
  const int share = a.H / a.Hkv;
  auto head_of = [&](int g, int loop) { return g * share + loop; };
  volatile int zero = 0;
  WaitCtx dc{&zero, nullptr, 100000000ull};

  if (warp == 0) {
    if (lane == 0) {
      // -------------------------------------------------------------- Q and dO
      const uint64_t keep = l2_policy_evict_last();
      uint32_t t1 = 0, t2 = 0;
      bool ok = true;
      while (ok && feed.next<false>(u, wc)) {
#pragma unroll 1
        for (int loop = 0; loop < loops && ok; ++loop) {
          const int h = head_of(u.g, loop);
#pragma unroll 1
          for (int tok = u.q0; tok < u.q1; tok += xg.tokens) {
            const uint32_t s1 = t1 % 3, s2 = t2 % 2;
            if (!wait_for(&y1_empty[s1], ((t1 / 3) & 1) ^ 1, wc)) { ok = false; break; }
            if (a.withhold && t1 == 0) { ok = false; break; }  // test hook: this tile never comes
            load_tile<DH>(&m.q, m.qv, &y1_full[s1], smem + P::kY1 + s1 * P::T, xg.r, h, tok, keep);
            ++t1;
            // A tile comes in when the products of the tile before last are
            // done, and is needed some 2,000 cycles later: from L2 it is there.
            if (tok + 3 * xg.tokens < u.q1) {
              prefetch_tile<DH>(&m.q, m.qv, xg.r, h, tok + 3 * xg.tokens);
              prefetch_tile<DH>(&m.dout, m.dv, xg.r, h, tok + 3 * xg.tokens);
            }
            if (!wait_for(&y2_empty[s2], ((t2 / 2) & 1) ^ 1, wc)) { ok = false; break; }
            load_tile<DH>(&m.dout, m.dv, &y2_full[s2], smem + P::kY2 + s2 * P::T, xg.r, h, tok, keep);
            ++t2;
          }
        }
      }
      for (uint32_t s = 0; s < 3; ++s)
        if (s < t1) wait_for(&y1_full[s], ((t1 - 1 - s) / 3) & 1, dc);
      for (uint32_t s = 0; s < 2; ++s)
        if (s < t2) wait_for(&y2_full[s], ((t2 - 1 - s) / 2) & 1, dc);
    }
  } else if (warp == 3) {
    // ---------------------------------------------------------------- units, their K and V tiles
    const WaitCtx wu = unit_wait(wc);
    const uint64_t once = l2_policy_evict_first();
    uint32_t n = 0;
    Walk it(a, xg, kTile, true);
    while (true) {
      int place;
      const bool more = it.next(u, place);
      u.k0 += place * kTile;
      take_share(u.q0, u.q1, xg.tokens, u.split, xg.splits);
      int go = 1;
      if (lane == 0) {
        go = feed.put(u, more ? 1 : 0, wu);
        if (go && more && u.q1 > u.q0) {
          go = wait_for(x_empty, (n & 1) ^ 1, wu);
          if (go) {
            // both tiles on one barrier: the second's bytes are added before the first phase can complete
            mbar_expect_tx(x_full, 2 * P::T);
#pragma unroll
            for (int c = 0; c < DH / 64; ++c) {
              tma_load_2d_hint(&m.k, x_full, smem + P::kX1 + c * P::kChunk, u.g * m.kv.x + c * 64, u.g * m.kv.y + u.k0, once);
              tma_load_2d_hint(&m.v, x_full, smem + P::kX2 + c * P::kChunk, u.g * m.vv.x + c * 64, u.g * m.vv.y + u.k0, once);
            }
            ++n;
          }
        }
      }
      if (!__shfl_sync(0xffffffffu, go, 0) || !more) break;
    }
    if (lane == 0 && n > 0) wait_for(x_full, (n - 1) & 1, dc);
  } else if (warp == 2) {
    // ---------------------------------------------------------------- rows past the last query; lse and D
    uint32_t t = 0;
    bool ok = true;
    while (ok) {
      int w = 1;
      if (lane == 0) w = feed.next<false>(u, wc);
      if (!__shfl_sync(0xffffffffu, w, 0)) break;
      const int q0 = __shfl_sync(0xffffffffu, u.q0, 0), q1 = __shfl_sync(0xffffffffu, u.q1, 0),
                g = __shfl_sync(0xffffffffu, u.g, 0);
      float lv[4], dv[4];
      auto fetch = [&](int loop, int tok) {
        const int rows = min(q1 - tok, xg.tokens) << xg.log2r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = lane + 32 * i;
          const int64_t at = (int64_t)(head_of(g, loop) + (r & (xg.r - 1))) * a.N + tok + (r >> xg.log2r);
          lv[i] = r < rows ? neg_lse_log2(a.lse[at]) : -INFINITY;
          dv[i] = r < rows ? -a.dsum[at] : 0.0f;
        }
      };
#pragma unroll 1
      for (int loop = 0; loop < loops && ok; ++loop) {
#pragma unroll 1
        for (int tok0 = q0; tok0 < q1; tok0 += xg.tokens, ++t) {
          const uint32_t s1 = t % 3, s2 = t % 2;
          const int valid = min(q1 - tok0, xg.tokens) << xg.log2r;
          if (tok0 == q0) fetch(loop, tok0);
          if (lane == 0) w = wait_for(&y1_full[s1], (t / 3) & 1, wc);
          if (!__shfl_sync(0xffffffffu, w, 0)) { ok = false; break; }
          __syncwarp();
          zero_rows<DH>(smem + P::kY1 + s1 * P::T, valid, lane);
#pragma unroll
          for (int i = 0; i < 4; ++i) vec1[s1 * kTile + lane + 32 * i] = lv[i];
          __syncwarp();
          float nv[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) nv[i] = dv[i];
          if (lane == 0) mbar_arrive(&y1_ready[s1]);
          // the next tile's, before the wait for this one's dO
          if (tok0 + xg.tokens < q1) fetch(loop, tok0 + xg.tokens);
          if (lane == 0) w = wait_for(&y2_full[s2], (t / 2) & 1, wc);
          if (!__shfl_sync(0xffffffffu, w, 0)) { ok = false; break; }
          __syncwarp();
          zero_rows<DH>(smem + P::kY2 + s2 * P::T, valid, lane);
#pragma unroll
          for (int i = 0; i < 4; ++i) vec2[s2 * kTile + lane + 32 * i] = nv[i];
          __syncwarp();
          if (lane == 0) mbar_arrive(&y2_ready[s2]);
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- products
    const bool leader = elect_one();
    const uint32_t x1_lo = desc_lo(smem_u32(smem + P::kX1), 16), x2_lo = desc_lo(smem_u32(smem + P::kX2), 16),
                   y1_lo = desc_lo(smem_u32(smem + P::kY1), 16), y2_lo = desc_lo(smem_u32(smem + P::kY2), 16),
                   y1t_lo = desc_lo(smem_u32(smem + P::kY1), P::kChunk), y2t_lo = desc_lo(smem_u32(smem + P::kY2), P::kChunk);
    uint32_t t = 0, un = 0;
    bool ok = true;
    while (ok && feed.next<true>(u, wc)) {
      if (u.q1 <= u.q0) continue;
      const int per = (u.q1 - u.q0 + xg.tokens - 1) / xg.tokens, n = per * loops;
      if (!wait_for(x_full, un & 1, wc)) break;
      int left = u.q1 - u.q0, open = 0;  // tokens from this tile on in its loop; rows of tile t - 1 (0: none)
#pragma unroll 1
      for (int j = 0; j <= n; ++j) {
        if (j < n) {
          // S^T(t) goes where dP^T(t - 1) was
          ok = wait_for(&y1_ready[t % 3], (t / 3) & 1, wc) && (t == 0 || wait_for(dp_free, (t - 1) & 1, wc));
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            issue_nt<DH>(tS(t), x1_lo, y1_lo + (t % 3) * (P::T >> 4));
            umma_commit(s_full);
          }
        }
        if (open > 0) {
          // dV and dK of tile t - 1
          const uint32_t tp = t - 1;
          ok = wait_for(&p_full[tp & 1], (tp >> 1) & 1, wc) && (j > 1 || un == 0 || wait_for(acc_empty, (un - 1) & 1, wc));
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            issue_acc<DH>(tV, tS(tp), y2t_lo + (tp % 2) * (P::T >> 4), open, j > 1);
            issue_acc<DH>(tK, tS(tp) + 32, y1t_lo + (tp % 3) * (P::T >> 4), open, j > 1);
            umma_commit(&y1_empty[tp % 3]);
            umma_commit(&y2_empty[tp % 2]);
            if (j == n) umma_commit(acc_full);
          }
        }
        if (j < n) {
          // dP^T(t) goes where dV and dK of tile t - 1 read P and dS
          ok = wait_for(&y2_ready[t % 2], (t / 2) & 1, wc);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            issue_nt<DH>(tD(t), x2_lo, y2_lo + (t % 2) * (P::T >> 4));
            umma_commit(d_full);
            if (j + 1 == n) umma_commit(x_empty);
          }
          open = min(left, xg.tokens) << xg.log2r;
          left -= xg.tokens;
          if (left <= 0) left = u.q1 - u.q0;
          ++t;
        }
      }
      ++un;
    }
    if (leader) umma_commit(done_bar);
    wait_for(done_bar, 0, dc);
  } else if (warp < 12) {
    // ---------------------------------------------------------------- P and dS
    const int wg = (warp - 4) >> 2, sub = warp & 3;
    const uint32_t at = ((uint32_t)(sub * 32) << 16) + 64 * wg;
    const float scale_log2 = kLog2e * rsqrtf((float)DH);
    uint32_t t = 0;
    bool ok = true;
    while (ok && feed.next<true>(u, wc)) {
      const int n = u.q1 > u.q0 ? (u.q1 - u.q0 + xg.tokens - 1) / xg.tokens * loops : 0;
#pragma unroll 1
      for (int j = 0; j < n; ++j, ++t) {
        ok = wait_for(s_full, t & 1, wc) && wait_for(&y1_ready[t % 3], (t / 3) & 1, wc);
        if (!ok) break;
        tc_fence_after();
        const uint32_t ts = tS(t) + at;
        const ulonglong2* nl = reinterpret_cast<const ulonglong2*>(vec1 + (t % 3) * kTile + 64 * wg);
        float p[64];
        tmem_ld32(ts, p);
        tmem_ld32(ts + 32, p + 32);
        tmem_ld_wait();
        // Columns past the last query: zeroed rows of Q and -inf make P 0.
        const uint64_t sc2 = f2_pack(scale_log2, scale_log2);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const ulonglong2 v = nl[e];  // four columns
          exp2_pair(p + 4 * e, sc2, v.x);
          exp2_pair(p + 4 * e + 2, sc2, v.y);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) pk[e] = pack_bf16x2(p[32 * c + 2 * e], p[32 * c + 2 * e + 1]);
          tmem_st16u(ts + 16 * c, pk);
        }
        ok = wait_for(d_full, t & 1, wc) && wait_for(&y2_ready[t % 2], (t / 2) & 1, wc);
        if (!ok) break;
        tc_fence_after();
        const ulonglong2* dd = reinterpret_cast<const ulonglong2*>(vec2 + (t % 2) * kTile + 64 * wg);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float d[32];
          tmem_ld32(tD(t) + at + 32 * c, d);
          tmem_ld_wait();
          if (c == 1) {
            tc_fence_before();
            mbar_arrive(dp_free);
          }
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const ulonglong2 v = dd[8 * c + e];
            pk[2 * e] = ds_pair(p + 32 * c + 4 * e, d + 4 * e, v.x);
            pk[2 * e + 1] = ds_pair(p + 32 * c + 4 * e + 2, d + 4 * e + 2, v.y);
          }
          tmem_st16u(ts + 32 + 16 * c, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_full[t & 1]);
      }
    }
  } else {
    // ---------------------------------------------------------------- the results
    const WaitCtx wu = unit_wait(wc);
    const int sub = warp & 3, row = sub * 32 + lane;
    const uint32_t lanes = (uint32_t)(sub * 32) << 16;
    const int64_t rows = a.L * a.Hkv;
    uint32_t on = 0;
    while (feed.next<true, 500>(u, wu)) {
      const bool some = u.q1 > u.q0;
      if (some) {
        if (!wait_for<500>(acc_full, on & 1, wu)) break;
        ++on;
        tc_fence_after();
      }
      const int key = u.k0 + row;
      const bool live = key < u.k1;
      const int64_t o = live ? ((int64_t)key * a.Hkv + u.g) * DH : 0;
      float* pv = part ? part + ((int64_t)u.split * 2 * rows) * DH + o : nullptr;
      write_row<DH>(tV + lanes, 1.0f, some, live, static_cast<__nv_bfloat16*>(a.dv) + o, pv);
      write_row<DH>(tK + lanes, rsqrtf((float)DH), some, live, static_cast<__nv_bfloat16*>(a.dk) + o,
                    part ? pv + rows * DH : nullptr);
      if (some) {
        tc_fence_before();
        mbar_arrive(acc_empty);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The sum of the shares' rows, for rows of a segment: of dQ ([N, H], one
// tensor a share), or of dV and dK ([L, H_kv], two; blockIdx.y picks one).
// blockDim.y threads (up to eight) share a row's piece, each every
// blockDim.y-th share, in a fixed order.
template <int DH>
__global__ void __launch_bounds__(256) cross_sum_kernel(const CrossArgs a, bool keys, int splits,
                                                        const float* __restrict__ part) {
  __shared__ float4 lane_sum[256][2];
  if (!segments_ok(a, nullptr)) return;
  const int heads = keys ? a.Hkv : a.H;
  const int64_t pieces = (keys ? a.L : a.N) * heads * (DH / 8);
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t row = i / (DH / 8) / heads;
  bool inside = i < pieces;
  if (!keys) {
    if (a.q_off) inside = inside && row >= a.q_off[0] && row < a.q_off[a.S];
  } else if (inside && (a.kv_off || a.kv_len)) {
    int lo = 0, hi = a.S - 1;  // the last segment that starts at or before the row
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (segment(a, mid).k0 <= row) lo = mid; else hi = mid - 1;
    }
    const Seg s = segment(a, lo);
    inside = row >= s.k0 && row < s.k1;
  }
  const int64_t step = pieces * 8 * (keys ? 2 : 1);
  const float* p = part + (int64_t)blockIdx.y * pieces * 8 + i * 8;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
  if (inside) {
#pragma unroll 4
    for (int s = threadIdx.y; s < splits; s += blockDim.y) {
      const float4 u = *reinterpret_cast<const float4*>(p + s * step), v = *reinterpret_cast<const float4*>(p + s * step + 4);
      x.x += u.x, x.y += u.y, x.z += u.z, x.w += u.w;
      y.x += v.x, y.y += v.y, y.z += v.z, y.w += v.w;
    }
  }
  const int me = threadIdx.y * blockDim.x + threadIdx.x;
  lane_sum[me][0] = x;
  lane_sum[me][1] = y;
  __syncthreads();
  if (threadIdx.y != 0 || !inside) return;
  for (int k = 1; k < (int)blockDim.y; ++k) {
    const float4 u = lane_sum[me + k * blockDim.x][0], v = lane_sum[me + k * blockDim.x][1];
    x.x += u.x, x.y += u.y, x.z += u.z, x.w += u.w;
    y.x += v.x, y.y += v.y, y.z += v.z, y.w += v.w;
  }
  void* out = !keys ? a.dq : blockIdx.y ? a.dk : a.dv;
  static_cast<uint4*>(out)[i] = make_uint4(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w), pack_bf16x2(y.x, y.y),
                                           pack_bf16x2(y.z, y.w));
}

// Shares of the keys for dQ, as in the forward.
int dq_splits(int64_t N, int64_t L, int H, int r, int S) {
  return shares(places_most(N, kTile / r, S) * (H / r), ceil_div(L, S), kTile, kSplitSms);
}
// Shares of the queries for dK and dV.  One segment makes equal units: of one
// to four rounds over the SMs the first that leaves under a twentieth of them
// idle, else the fullest (48 units: 3 shares, 144 of 148 SMs).  Ragged
// segments take four rounds, so that the last one's ragged end costs little.
int dkv_splits(int64_t N, int64_t L, int H_kv, int r, int S) {
  const int64_t units = places_most(L, kTile, S) * H_kv;
  int64_t rounds = 4;
  if (S == 1 && units > 0) {
    double best = 0.0;
    for (int64_t k = 1; k <= 4 && best < 0.95; ++k) {
      const int64_t sms = k * kSplitSms, n = sms / units;
      const double used = (double)(n * units) / (double)sms;
      if (used > best + 1e-9) best = used, rounds = k;
    }
  }
  return shares(units, ceil_div(N, S), kTile / r, rounds * kSplitSms);
}

struct BwdWs {
  size_t dsum, dq, dkv, total;
};
BwdWs bwd_ws(int64_t N, int64_t L, int H, int H_kv, int d_h, int S, int r) {
  BwdWs w{};
  const int nq = dq_splits(N, L, H, r, S), nk = dkv_splits(N, L, H_kv, r, S);
  w.dq = align_up((size_t)N * H * 4, 256);
  w.dkv = w.dq + align_up(nq > 1 ? (size_t)nq * N * H * d_h * 4 : 0, 256);
  w.total = w.dkv + (nk > 1 ? (size_t)nk * 2 * L * H_kv * d_h * 4 : 0);
  return w;
}

template <int DH>
cudaError_t launch_bwd(const DevCtx& c, CrossArgs a, uint8_t* ws, int* launches) {
  using P = BPlan<DH>;
  BMaps m{};
  const int r = pack_of(a);
  const int64_t HD = (int64_t)a.H * DH;
  const XGrid base = pack_grid(r);
  const BwdWs w = bwd_ws(a.N, a.L, a.H, a.Hkv, DH, a.S, r);
  a.dsum = reinterpret_cast<float*>(ws + w.dsum);
  bool ok = view_2d(&m.k, &m.kv, a.k, a.k_sn, a.k_sh, a.L, a.Hkv, DH) &&
            view_2d(&m.v, &m.vv, a.v, a.v_sn, a.v_sh, a.L, a.Hkv, DH);
  if (r > 1)
    ok = ok && make_tmap_heads(&m.q, a.q, DH, a.H, a.N, a.q_sh, a.q_sn, r, base.tokens) &&
         make_tmap_heads(&m.dout, a.dout, DH, a.H, a.N, DH, HD, r, base.tokens) &&
         make_tmap_heads(&m.out, a.out, DH, a.H, a.N, DH, HD, r, base.tokens);
  else
    ok = ok && view_2d(&m.q, &m.qv, a.q, a.q_sn, a.q_sh, a.N, a.H, DH) &&
         view_2d(&m.dout, &m.dv, a.dout, HD, DH, a.N, a.H, DH) &&
         view_2d(&m.out, &m.dv, a.out, HD, DH, a.N, a.H, DH);
  if (!ok) return cudaErrorInvalidValue;
  cudaError_t e;
  if ((e = cudaFuncSetAttribute(cross_dq_kernel<DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::kBytes)) != cudaSuccess ||
      (e = cudaFuncSetAttribute(cross_dkv_kernel<DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::kBytes)) != cudaSuccess)
    return e;
  auto sum = [&](bool keys, int splits, const float* part) {
    const int64_t n = (keys ? a.L * a.Hkv : a.N * a.H) * (DH / 8);
    const int ny = splits >= 8 ? 8 : splits >= 4 ? 4 : 2;
    cross_sum_kernel<DH><<<dim3((unsigned)ceil_div(n, 256 / ny), keys ? 2 : 1), dim3(256 / ny, ny), 0, c.stream>>>(
        a, keys, splits, part);
    ++*launches;
    return cudaGetLastError();
  };
  if (a.N > 0) {
    XGrid x = base;
    x.heads = a.H / r;
    x.splits = dq_splits(a.N, a.L, a.H, r, a.S);
    float* part = x.splits > 1 ? reinterpret_cast<float*>(ws + w.dq) : nullptr;
    const int64_t grid = std::min<int64_t>(places_most(a.N, x.tokens, a.S) * x.heads * x.splits, c.num_sms);
    set_steps(&x, grid);
    cross_dq_kernel<DH><<<(unsigned)grid, kXThreads, P::kBytes, c.stream>>>(m, a, x, part, c.status,
                                                                          (unsigned long long)c.wait_ns);
    ++*launches;
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (part && (e = sum(false, x.splits, part)) != cudaSuccess) return e;
  }
  if (a.L > 0) {
    XGrid x = base;
    x.heads = a.Hkv;
    x.splits = dkv_splits(a.N, a.L, a.Hkv, r, a.S);
    float* part = x.splits > 1 ? reinterpret_cast<float*>(ws + w.dkv) : nullptr;
    const int64_t grid = std::min<int64_t>(places_most(a.L, kTile, a.S) * x.heads * x.splits, c.num_sms);
    set_steps(&x, grid);
    cross_dkv_kernel<DH><<<(unsigned)grid, kXThreads, P::kBytes, c.stream>>>(m, a, x, part, c.status,
                                                                           (unsigned long long)c.wait_ns);
    ++*launches;
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (part && (e = sum(true, x.splits, part)) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t cross_bwd_ws_bytes(int64_t N, int64_t L, int H, int H_kv, int d_h, int S) {
  // Packed or not is known with the strides only: the larger of the two.
  size_t most = 0;
  for (int r : {1, H / H_kv}) {
    if (r < 1 || r > 64 || (r & (r - 1))) continue;
    most = std::max(most, bwd_ws(N, L, H, H_kv, d_h, S, r).total);
  }
  return most;
}

cudaError_t launch_cross_bwd(const DevCtx& c, const CrossArgs& a, uint8_t* ws, int* launches) {
  *launches = 0;
  return a.d_h == 128 ? launch_bwd<128>(c, a, ws, launches) : launch_bwd<64>(c, a, ws, launches);
}

}  // namespace moga

// What the cross-attention kernels share: segments, the ring that hands work
// units to a CTA's roles, bounded waits, and tensor-core issue with short
// descriptor arithmetic.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"

namespace moga {
namespace {

constexpr int kXThreads = 512;
constexpr int kSplitSms = 148;  // a B200's SMs

// Segments of a call, read from device memory and checked there.
struct Seg {
  int q0, q1, k0, k1;
};
__device__ __forceinline__ Seg segment(const CrossArgs& a, int s) {
  Seg g;
  g.q0 = a.q_off ? a.q_off[s] : 0;
  g.q1 = a.q_off ? a.q_off[s + 1] : (int)a.N;
  g.k0 = a.kv_off ? a.kv_off[s] : 0;
  g.k1 = a.kv_off ? a.kv_off[s + 1] : (int)a.L;
  if (a.kv_len) g.k1 = a.kv_len[s] < 0 || a.kv_len[s] > g.k1 - g.k0 ? -1 : g.k0 + a.kv_len[s];
  return g;
}
// Offsets must rise from 0 or more to at most the rows there are, and a
// length must fit its segment.  Every thread of the block gets the answer.
__device__ __forceinline__ bool segments_ok(const CrossArgs& a, int* status) {
  bool bad = false;
#pragma unroll 1
  for (int s = threadIdx.x; s < a.S; s += blockDim.x) {
    const Seg g = segment(a, s);
    bad |= g.q0 < 0 || g.q1 < g.q0 || g.q1 > a.N || g.k0 < 0 || g.k1 < g.k0 || g.k1 > a.L;
    if (a.kv_off) bad |= a.kv_off[s + 1] < a.kv_off[s] || a.kv_off[s + 1] > a.L;
  }
  if (!__syncthreads_or(bad)) return true;
  if (threadIdx.x == 0 && status) atomicOr(status, DEV_RANGE);
  return false;
}

// The bounded wait of ptx.cuh, its loop out of line.  What runs here has to
// fit the instruction cache: with that one inlined at some twenty places the
// kernel had 114 KB of instructions, and a role's code was fetched anew each
// time it came round (187,200 x 512 keys: 745 us; 613 us with 45 KB).
template <int kSleep>
__device__ __noinline__ bool wait_more(uint32_t bar, uint32_t parity, const WaitCtx c) {
  uint32_t n = 0, t0 = 0;
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if (kSleep > 0) __nanosleep(kSleep);
    if (++n & 63u) continue;
    const uint32_t t = (uint32_t)(global_timer_ns() >> 10);  // about a microsecond
    if (n == 64) t0 = t;
    if (t - t0 > (uint32_t)min((unsigned long long)(c.limit_ns >> 10), 0xfffffffeull)) {
      *c.abort_flag = 1;
      if (c.status) atomicOr(c.status, DEV_TIMEOUT);
    }
    if (*c.abort_flag) return false;
  }
}
template <int kSleep = 0>
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, const WaitCtx& c) {
  return mbar_try_wait(bar, parity) || wait_more<kSleep>(smem_u32(bar), parity, c);
}

// For waits that last as long as a unit does (the writers of its results, the
// walk, which is a unit ahead, and warps that a unit has no rows for): the roles that step through the unit bound
// it, and their abort flag ends these too.
__device__ __forceinline__ WaitCtx unit_wait(WaitCtx c) {
  c.limit_ns = c.limit_ns < (1ull << 33) ? c.limit_ns * 256 : c.limit_ns;
  return c;
}

__device__ __forceinline__ void tmem_st1(uint32_t taddr, float v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(__float_as_uint(v)) : "memory");
}

// The products with descriptors of 128-byte swizzled operands (8-row groups
// 1,024 bytes apart) given by their low words: the high word is a constant.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | ((lbo >> 4) << 16); }
__device__ __forceinline__ void umma_lo(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void umma_ts_lo(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}\n" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(acc), "n"(kDescHi)
      : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok));
  return ok != 0;
}

// mbar_try_wait without its suspension.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

struct XUnit {
  int g;               // key head, or query head without packing
  int q0, q1;          // this unit's first token and the end of its tokens
  int k0, k1;          // its first key and the end of its keys
  int split;           // its share of a long range
};

struct XGrid {
  int tokens;          // tokens of a query tile: 128 / r
  int r, log2r;        // query heads of a tile
  int heads;           // units of a place
  int splits;          // shares of the keys (forward, dQ) or of the queries (dK, dV)
  int step_w, step_g;  // a step of gridDim.x units, in places and shares, and in heads
};

constexpr int kFeedSlots = 4;
// One thread each for K/V or X/Y loads, products, and rows past a segment's
// end; 12 warps of softmax and epilogue.
constexpr int kFeedReaders = 15;

// One warp walks a CTA's units and hands each to the other roles through a
// ring in shared memory: with the walk in every role the code that runs did
// not fit the instruction cache.
struct Feed {
  int4* ring;          // [kFeedSlots][2]: (g, q0, q1, split), (k0, k1, flag: 0 at the end, -)
  uint64_t* full;
  uint64_t* empty;
  uint32_t n;
  // The next unit; false: none is left, or a wait gave up.  `warp`: all of a
  // warp's threads read, and its first one frees the slot.
  template <bool kWarp, int kSleep = 0>
  __device__ __forceinline__ bool next(XUnit& u, const WaitCtx& wc) {
    return next_flag<kWarp, kSleep>(u, wc) != 0;
  }
  template <bool kWarp, int kSleep = 0>
  __device__ __forceinline__ int next_flag(XUnit& u, const WaitCtx& wc) {
    const uint32_t s = n % kFeedSlots;
    if (!wait_for<kSleep>(&full[s], (n / kFeedSlots) & 1, wc)) return false;
    const int4 a = ring[2 * s], b = ring[2 * s + 1];
    if (kWarp) __syncwarp();
    if (!kWarp || (threadIdx.x & 31) == 0) mbar_arrive(&empty[s]);
    ++n;
    u = XUnit{a.x, a.y, a.z, b.x, b.y, a.w};
    return b.z;
  }
  __device__ __forceinline__ bool put(const XUnit& u, int more, const WaitCtx& wc) {
    const uint32_t s = n % kFeedSlots;
    if (!wait_for(&empty[s], ((n / kFeedSlots) & 1) ^ 1, wc)) return false;
    ring[2 * s] = make_int4(u.g, u.q0, u.q1, u.split);
    ring[2 * s + 1] = make_int4(u.k0, u.k1, more, 0);
    mbar_arrive(&full[s]);
    ++n;
    return true;
  }
};

// A CTA's units are blockIdx.x, then every gridDim.x-th, the heads of a place
// next to one another (CTAs that run at once read whole token rows).  A place
// is `per` queries or keys of a segment.  A whole warp walks, each lane
// holding one of 32 segments, and carries head and place along: dividing them
// out of an index for every unit took some 3,000 cycles.
struct Walk {
  const CrossArgs& a;
  const XGrid& x;
  int per;
  bool by_keys;
  int g, w;            // head; place and share
  int chunk, before;   // first of the 32 segments, places before them
  Seg seg;             // this lane's segment
  int n, incl, all;    // its places, with those of the lanes below, of all lanes
  __device__ __forceinline__ Walk(const CrossArgs& a_, const XGrid& x_, int per_, bool by_keys_)
      : a(a_), x(x_), per(per_), by_keys(by_keys_), chunk(0), before(0) {
    w = (int)blockIdx.x / x.heads;
    g = (int)blockIdx.x - w * x.heads;
    load();
  }
  __device__ __forceinline__ void load() {
    const int lane = threadIdx.x & 31;
    seg = Seg{0, 0, 0, 0};
    if (chunk + lane < a.S) seg = segment(a, chunk + lane);
    if (a.S > 1) {
      // The 32 segments by the length of their units, longest first: units
      // are dealt in turn, and the last, partial round is then of short ones.
      // Every other 32 the other way, so that long ones do not meet long ones.
      const int len = by_keys ? seg.q1 - seg.q0 : seg.k1 - seg.k0, cost = (chunk & 32) ? -len : len;
      int rank = 0, src = lane;
#pragma unroll 4
      for (int j = 0; j < 32; ++j) {
        const int c = __shfl_sync(0xffffffffu, cost, j);
        rank += c > cost || (c == cost && j < lane);
      }
#pragma unroll 4
      for (int j = 0; j < 32; ++j)
        if (__shfl_sync(0xffffffffu, rank, j) == lane) src = j;
      seg = Seg{__shfl_sync(0xffffffffu, seg.q0, src), __shfl_sync(0xffffffffu, seg.q1, src),
                __shfl_sync(0xffffffffu, seg.k0, src), __shfl_sync(0xffffffffu, seg.k1, src)};
    }
    n = ((by_keys ? seg.k1 - seg.k0 : seg.q1 - seg.q0) + per - 1) / per;
    // Queries without keys are no units (empty_segments sets their rows): the
    // issuing warp looks for the next unit with keys before it has finished
    // this one, and would wait for ever behind a ring full of others.  With
    // shares a CTA has one unit, and the join wants a word from each.
    if (!by_keys && x.splits == 1 && seg.k1 <= seg.k0) n = 0;
    incl = n;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, m);
      if (lane >= m) incl += t;
    }
    all = __shfl_sync(0xffffffffu, incl, 31);
  }
  // The next unit with its whole segment in q0..k1, and its place in the
  // segment; false: none is left.
  __device__ __forceinline__ bool next(XUnit& u, int& place) {
    int p = w;
    u.split = 0;
    if (x.splits > 1) {
      p = (int)((unsigned)w / (unsigned)x.splits);
      u.split = w - p * x.splits;
    }
    while (p >= before + all) {
      before += all;
      chunk += 32;
      if (chunk >= a.S) return false;
      load();
    }
    const unsigned mask = __ballot_sync(0xffffffffu, incl > p - before);
    const int src = __ffs(mask) - 1;
    place = p - before - __shfl_sync(0xffffffffu, incl - n, src);
    u.g = g;
    u.q0 = __shfl_sync(0xffffffffu, seg.q0, src);
    u.q1 = __shfl_sync(0xffffffffu, seg.q1, src);
    u.k0 = __shfl_sync(0xffffffffu, seg.k0, src);
    u.k1 = __shfl_sync(0xffffffffu, seg.k1, src);
    w += x.step_w;
    g += x.step_g;
    if (g >= x.heads) {
      g -= x.heads;
      ++w;
    }
    return true;
  }
};

// Share `split` of [lo, hi) in tiles of `tile`: the first shares have one more.
__device__ __forceinline__ void take_share(int& lo, int& hi, int tile, int split, int splits) {
  if (splits < 2) return;
  const unsigned n = (unsigned)(hi - lo + tile - 1) / (unsigned)tile, each = n / (unsigned)splits,
                 over = n - each * (unsigned)splits, s = (unsigned)split;
  const int first = lo + (int)((each * s + min(s, over)) * (unsigned)tile);
  hi = min(hi, first + (int)((each + (s < over ? 1u : 0u)) * (unsigned)tile));
  lo = min(first, hi);
}

// Head h's rows in a 2-D view of a [n, heads, d_h] tensor: column h * x + c,
// row h * y + token (token-major: y = 0; head-major: x = 0).
struct XView {
  int x, y;
};

// Query rows of no segment (before the first and behind the last): 0, and
// lse = -inf where it is given.  One thread of `threads` in the grid.
template <int DH>
__device__ __forceinline__ void fill_rows(const CrossArgs& a, void* out, float* lse, int64_t thread, int64_t threads) {
  if (!a.fill || !a.q_off) return;
  const int64_t lo = a.q_off[0], hi = a.q_off[a.S], n = lo + a.N - hi;
  for (int64_t i = thread; i < n * a.H * (DH / 8); i += threads) {
    const int64_t r = i / (DH / 8) / a.H, tok = r < lo ? r : r - lo + hi;
    const int64_t rest = i - r * a.H * (DH / 8);
    static_cast<uint4*>(out)[tok * a.H * (DH / 8) + rest] = make_uint4(0, 0, 0, 0);
    if (lse && rest % (DH / 8) == 0) lse[rest / (DH / 8) * a.N + tok] = -INFINITY;
  }
}

// Refused segments: NaN in every row of an output that is to be filled.  All
// threads of the grid; out of line, since what a small call fetches counts.
__device__ __noinline__ void refuse_rows(void* out, float* lse, int64_t rows, int pieces) {
  const int64_t first = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, step = (int64_t)gridDim.x * blockDim.x;
  const uint32_t nan2 = 0x7fc07fc0u;  // two bf16 NaN
  for (int64_t i = first; i < rows * pieces; i += step) static_cast<uint4*>(out)[i] = make_uint4(nan2, nan2, nan2, nan2);
  if (lse)
    for (int64_t i = first; i < rows; i += step) lse[i] = __int_as_float(0x7fc00000);
}

// The rows of segments without keys: 0, and lse = -inf where it is given.
// One warp of `warps` in the grid.
template <int DH>
__device__ __forceinline__ void empty_segments(const CrossArgs& a, void* out, float* lse, int64_t warp, int64_t warps) {
  const int lane = threadIdx.x & 31;
  for (int base = 0; base < a.S; base += 32) {
    Seg g{0, 0, 0, 0};
    if (base + lane < a.S) g = segment(a, base + lane);
    unsigned empty = __ballot_sync(0xffffffffu, g.q1 > g.q0 && g.k1 <= g.k0);
    for (; empty; empty &= empty - 1) {
      const int src = __ffs(empty) - 1;
      const int q0 = __shfl_sync(0xffffffffu, g.q0, src), q1 = __shfl_sync(0xffffffffu, g.q1, src);
      for (int64_t tok = q0 + warp; tok < q1; tok += warps) {
        uint4* row = static_cast<uint4*>(out) + tok * a.H * (DH / 8);
        for (int i = lane; i < a.H * (DH / 8); i += 32) row[i] = make_uint4(0, 0, 0, 0);
        if (lse)
          for (int h = lane; h < a.H; h += 32) lse[(int64_t)h * a.N + tok] = -INFINITY;
      }
    }
  }
}

// One operand tile: 128 rows of one head (2-D view), or 128 / r tokens of r heads (3-D).
template <int DH>
__device__ __forceinline__ void load_tile(const CUtensorMap* map, const XView& v, uint64_t* bar, uint8_t* dst, int r,
                                          int head, int row, uint64_t policy) {
  mbar_expect_tx(bar, kTile * DH * 2);
#pragma unroll
  for (int c = 0; c < DH / 64; ++c) {
    if (r > 1)
      tma_load_3d(map, bar, dst + c * kTile * 128, c * 64, head, row);
    else
      tma_load_2d_hint(map, bar, dst + c * kTile * 128, head * v.x + c * 64, head * v.y + row, policy);
  }
}

// The same tile into L2.
template <int DH>
__device__ __forceinline__ void prefetch_tile(const CUtensorMap* map, const XView& v, int r, int head, int row) {
#pragma unroll
  for (int c = 0; c < DH / 64; ++c) {
    if (r > 1)
      asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map), "r"(c * 64),
                   "r"(head), "r"(row)
                   : "memory");
    else
      asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map),
                   "r"(head * v.x + c * 64), "r"(head * v.y + row)
                   : "memory");
  }
}

// Zeroes rows [valid, next multiple of 16) of a tile (a whole warp).  Products
// run in steps of 16 rows, and what a row of another segment or past the last
// one holds may be NaN, of which 0 times is NaN.
template <int DH>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int valid, int lane) {
  if (valid >= kTile) return;
  const int end = min((valid + 15) & ~15, kTile);
#pragma unroll 1
  for (int i = lane; i < (end - valid) * (DH / 8); i += 32) {
    const int piece = i & 7, c = (i >> 3) % (DH / 64), r = valid + (i >> 3) / (DH / 64);
    *reinterpret_cast<uint4*>(tile + c * kTile * 128 + r * 128 + piece * 16) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// 2-D view of a [n, heads, d_h] tensor whose box is 64 columns x 128 tokens of a head.
inline bool view_2d(CUtensorMap* map, XView* v, const void* base, int64_t sn, int64_t sh, int64_t n, int H, int d_h) {
  if (n == 0) return true;  // nothing is read through it
  if (H == 1 || sn >= (H - 1) * sh + d_h) {  // token-major
    *v = XView{(int)sh, 0};
    return make_tmap_2d(map, base, (uint64_t)((H - 1) * sh + d_h), (uint64_t)n, (uint64_t)sn * 2, kTile);
  }
  *v = XView{0, (int)(sh / sn)};
  return make_tmap_2d(map, base, (uint64_t)d_h, (uint64_t)(H - 1) * (sh / sn) + n, (uint64_t)sn * 2, kTile);
}

// Query heads of a tile: all that share a key head, where they are a power of
// two up to 64 and q is token-major with a token stride in whole head strides.
inline int pack_of(const CrossArgs& a) {
  const int r = a.H / a.Hkv;
  if (a.N == 0 || r < 2 || r > 64 || (r & (r - 1))) return 1;
  return a.q_sn >= (a.H - 1) * a.q_sh + a.d_h && a.q_sn % a.q_sh == 0 ? r : 1;
}

inline void set_steps(XGrid* x, int64_t grid) {
  x->step_w = (int)(grid / x->heads);
  x->step_g = (int)(grid % x->heads);
}
inline XGrid pack_grid(int r) {
  XGrid x{};
  x.r = r;
  while (1 << x.log2r < r) ++x.log2r;
  x.tokens = kTile / r;
  return x;
}
// Places of `per` rows in n rows of S segments, at most: each may add a ragged one.
inline int64_t places_most(int64_t n, int64_t per, int64_t S) {
  return n == 0 ? 0 : ceil_div(n, per) + (S < n ? S : n) - 1;
}
// Shares of a range of `len` rows in tiles of `tile`, for `units` units without
// shares: as many as SMs allow, each of two tiles at least.
inline int shares(int64_t units, int64_t len, int64_t tile, int64_t sms) {
  if (units == 0 || units * 2 > sms) return 1;
  const int64_t n = sms / units, most = ceil_div(len, 2 * tile);
  return (int)(n < most ? n : most > 1 ? most : 1);
}

}  // namespace
}  // namespace moga

// Norm of every query and key head, with the rotation by the token's place in
// the same pass, and its gradients.
//
// For a token, a head x of d_h channels, a weight w and the pairs (a, b) of a
// head's channels:
//   r = 1 / sqrt(mean_c x_c^2 + eps),   z_c = w_c x_c r,
//   y_a = z_a cos t - z_b sin t,   y_b = z_a sin t + z_b cos t,
// with t the pair's angle at the token's position.  Backward, with dz the
// gradient dy turned by -t and n_c = x_c r:
//   dw_c = sum over tokens and heads of dz_c n_c,
//   dx_c = r (g_c - n_c mean_e(g_e n_e)),   g_c = dz_c w_c.
//
// Both kernels are bound by HBM: every input is read once and every output
// written once.  A lane owns eight channels of a head (a row takes 16 lanes
// at d_h = 128, 8 at 64), chosen so that it owns whole pairs in either
// pairing: eight consecutive channels, or four and the four half a head
// further.  The row sums are then three or four shuffles, and the rotation
// needs none.  A warp's item is one token and up to kRows rows per lane group
// of its query heads or of its key heads, all loaded before the first is
// used; the cosines and sines are read once for those rows.  Measured at
// 187,200 tokens of 24 heads, 128 channels, bf16 with rotation: forward 383 to 416 us
// (5.5 to 6.0 TB/s, 0.84 to 0.92 of the measured copy rate), gradients 608 to
// 633 us (5.5 to 5.7 TB/s); fp32 at 62,400 tokens: 204 and 313 us (5.6 and 6.1
// TB/s).  The register limits (64 forward, 128 gradients) cost the bf16 instances
// 4 to 16 bytes of spills a thread.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"

namespace moga {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormWarps = kNormThreads / 32;
// Rows of one lane group in flight: 64 bytes a lane and tensor (six rows cover
// 12 heads of 128 channels in one item).
template <typename T>
constexpr int kRows = sizeof(T) == 2 ? 6 : 3;

template <typename T>
struct Raw;  // eight channels as loaded
template <>
struct Raw<__nv_bfloat16> {
  uint2 lo, hi;
};
template <>
struct Raw<float> {
  float4 lo, hi;
};

// Channel of a lane's element e (0..7): whole pairs in either pairing.
template <int DH, bool kHalves>
__device__ __forceinline__ int channel(int l, int e) {
  return kHalves ? (e < 4 ? 4 * l + e : DH / 2 + 4 * l + e - 4) : 8 * l + e;
}

// Plain (not read-only) loads: the outputs may be the inputs themselves.
template <int DH, bool kHalves>
__device__ __forceinline__ void load8(Raw<__nv_bfloat16>& r, const __nv_bfloat16* p, int l) {
  if (kHalves) {
    r.lo = __ldcs(reinterpret_cast<const uint2*>(p + 4 * l));
    r.hi = __ldcs(reinterpret_cast<const uint2*>(p + DH / 2 + 4 * l));
  } else {
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p + 8 * l));
    r.lo = make_uint2(v.x, v.y);
    r.hi = make_uint2(v.z, v.w);
  }
}
template <int DH, bool kHalves>
__device__ __forceinline__ void load8(Raw<float>& r, const float* p, int l) {
  r.lo = __ldcs(reinterpret_cast<const float4*>(p + channel<DH, kHalves>(l, 0)));
  r.hi = __ldcs(reinterpret_cast<const float4*>(p + channel<DH, kHalves>(l, 4)));
}
__device__ __forceinline__ void unpack2(uint32_t u, float& a, float& b) {
  a = __uint_as_float(u << 16);
  b = __uint_as_float(u & 0xffff0000u);
}
__device__ __forceinline__ void values(const Raw<__nv_bfloat16>& r, float (&x)[8]) {
  unpack2(r.lo.x, x[0], x[1]);
  unpack2(r.lo.y, x[2], x[3]);
  unpack2(r.hi.x, x[4], x[5]);
  unpack2(r.hi.y, x[6], x[7]);
}
__device__ __forceinline__ void values(const Raw<float>& r, float (&x)[8]) {
  x[0] = r.lo.x, x[1] = r.lo.y, x[2] = r.lo.z, x[3] = r.lo.w;
  x[4] = r.hi.x, x[5] = r.hi.y, x[6] = r.hi.z, x[7] = r.hi.w;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
template <int DH, bool kHalves>
__device__ __forceinline__ void store8(__nv_bfloat16* p, int l, const float (&x)[8]) {
  const uint2 lo = make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3]));
  const uint2 hi = make_uint2(pack2(x[4], x[5]), pack2(x[6], x[7]));
  if (kHalves) {
    __stcs(reinterpret_cast<uint2*>(p + 4 * l), lo);
    __stcs(reinterpret_cast<uint2*>(p + DH / 2 + 4 * l), hi);
  } else {
    __stcs(reinterpret_cast<uint4*>(p + 8 * l), make_uint4(lo.x, lo.y, hi.x, hi.y));
  }
}
template <int DH, bool kHalves>
__device__ __forceinline__ void store8(float* p, int l, const float (&x)[8]) {
  __stcs(reinterpret_cast<float4*>(p + channel<DH, kHalves>(l, 0)), make_float4(x[0], x[1], x[2], x[3]));
  __stcs(reinterpret_cast<float4*>(p + channel<DH, kHalves>(l, 4)), make_float4(x[4], x[5], x[6], x[7]));
}

// Cosines and sines of a lane's four pairs at a token.  False when a listed
// position is outside the table (the token is then skipped).
template <bool kRot>
__device__ __forceinline__ bool angles(const NormArgs& a, int64_t n, int l, float (&c)[4], float (&s)[4], int* status) {
  if (!kRot) return true;
  int p0, p1, p2;
  if (a.pos) {
    const int32_t* p = a.pos + 3 * n;
    p0 = p[0], p1 = p[1], p2 = p[2];
    const bool bad = (a.end0 > 0 && (unsigned)p0 >= (unsigned)a.P) ||
                     (a.end1 > a.end0 && (unsigned)p1 >= (unsigned)a.P) ||
                     (a.end2 > a.end1 && (unsigned)p2 >= (unsigned)a.P);
    if (bad) {
      if (status) atomicOr(status, DEV_RANGE);
      return false;
    }
  } else {
    // token0 and n are below 2^31, so the sum fits 32 unsigned bits
    const uint32_t i = (a.token0 + (uint32_t)n) % a.cells;
    p0 = (int)(i / a.frame);
    const uint32_t rest = i - (uint32_t)p0 * a.frame;
    p1 = (int)(rest / a.width);
    p2 = (int)(rest - (uint32_t)p1 * a.width);
  }
  const float2* table = reinterpret_cast<const float2*>(a.table);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = 4 * l + i;
    const int p = j < a.end0 ? p0 : j < a.end1 ? p1 : p2;
    float2 t = make_float2(1.0f, 0.0f);  // pairs past the rotated ones
    if (j < a.end2) t = __ldg(table + (int64_t)p * a.half + j);
    c[i] = t.x;
    s[i] = t.y;
  }
  return true;
}

// Turns the pairs of x by the angles (sign = 1) or back (-1), two products at
// a time: (u, v) c + (-v, u) s, or over two pairs where a pair's channels are
// four elements apart.
template <bool kHalves>
__device__ __forceinline__ void turn(float (&x)[8], const float (&c)[4], const float (&s)[4], float sign) {
  if (kHalves) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const uint64_t u = f2_pack(x[i], x[i + 1]), v = f2_pack(x[i + 4], x[i + 5]);
      const uint64_t c2 = f2_pack(c[i], c[i + 1]), s2 = f2_pack(sign * s[i], sign * s[i + 1]);
      const uint64_t m2 = f2_pack(-sign * s[i], -sign * s[i + 1]);
      f2_unpack(f2_fma(v, m2, f2_mul(u, c2)), x[i], x[i + 1]);
      f2_unpack(f2_fma(u, s2, f2_mul(v, c2)), x[i + 4], x[i + 5]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u = x[2 * i], v = x[2 * i + 1];
      const uint64_t y = f2_mul(f2_pack(u, v), f2_pack(c[i], c[i]));
      f2_unpack(f2_fma(f2_pack(v, u), f2_pack(-sign * s[i], sign * s[i]), y), x[2 * i], x[2 * i + 1]);
    }
  }
}

// Eight values as four packed pairs.
struct Eight {
  uint64_t p[4];
  __device__ __forceinline__ explicit Eight(const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = f2_pack(x[2 * i], x[2 * i + 1]);
  }
  __device__ __forceinline__ void to(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) f2_unpack(p[i], x[2 * i], x[2 * i + 1]);
  }
};
__device__ __forceinline__ float dot8(const Eight& a, const Eight& b) {
  uint64_t t = f2_mul(a.p[0], b.p[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) t = f2_fma(a.p[i], b.p[i], t);
  float x, y;
  f2_unpack(t, x, y);
  return x + y;
}

// NaN in a lane group's rows (h0, h0 + step, ...) of a token that is skipped.
template <int DH, bool kHalves, typename T>
__device__ __forceinline__ void fill_nan(const NormArgs& a, int64_t n, int t, int l, int h0, int step) {
  const float x = __int_as_float(0x7fc00000);
  const float v[8] = {x, x, x, x, x, x, x, x};
  T* y = static_cast<T*>(a.y[t]) + n * a.heads[t] * DH;
#pragma unroll 1
  for (int u = 0, h = h0; u < a.rows[t] && h < a.heads[t]; ++u, h += step) store8<DH, kHalves>(y + h * DH, l, v);
}

// Sum over the lanes that share a row.
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int m = LPR / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// Walks a warp's items (token, chunk) with a fixed step, without dividing.
struct Items {
  int64_t n;
  int chunk, ipt;
  int64_t dn;
  int dc;
  __device__ __forceinline__ Items(int per_token) : ipt(per_token) {
    const int64_t w = (int64_t)blockIdx.x * kNormWarps + (threadIdx.x >> 5);
    const int64_t nw = (int64_t)gridDim.x * kNormWarps;
    n = w / ipt;
    chunk = (int)(w - n * ipt);
    dn = nw / ipt;
    dc = (int)(nw - dn * ipt);
  }
  __device__ __forceinline__ void next() {
    n += dn;
    chunk += dc;
    if (chunk >= ipt) {
      chunk -= ipt;
      ++n;
    }
  }
};

template <int DH, typename T, bool kHalves, bool kRot>
__global__ void __launch_bounds__(kNormThreads, 4) norm_rope_kernel(const NormArgs a, int* status) {
  constexpr int LPR = DH / 8, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, l = lane % LPR, grp = lane / LPR;
  for (Items it(a.chunks[0] + a.chunks[1]); it.n < a.N; it.next()) {
    const int t = it.chunk >= a.chunks[0];  // 0: query heads, 1: key heads
    const int h0 = (t ? it.chunk - a.chunks[0] : it.chunk) * a.rows[t] * RPW + grp;
    const T* x = static_cast<const T*>(a.x[t]) + it.n * a.sn[t];
    Raw<T> raw[kRows<T>];
#pragma unroll
    for (int u = 0; u < kRows<T>; ++u) {
      const int h = h0 + u * RPW;
      raw[u] = Raw<T>{};
      if (u < a.rows[t] && h < a.heads[t]) load8<DH, kHalves>(raw[u], x + h * a.sh[t], l);
    }
    float c[4], s[4];
    if (!angles<kRot>(a, it.n, l, c, s, status)) {
      if (a.fill) fill_nan<DH, kHalves, __nv_bfloat16>(a, it.n, t, l, h0, RPW);
      continue;
    }
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = a.w[t] ? __ldg(a.w[t] + channel<DH, kHalves>(l, e)) : 1.0f;
    const Eight w8(w);
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y[t]) + it.n * a.heads[t] * DH;
#pragma unroll
    for (int u = 0; u < kRows<T>; ++u) {
      if (u >= a.rows[t]) break;
      const int h = h0 + u * RPW;
      float v[8];
      values(raw[u], v);
      Eight x8(v);
      const float r = rsqrtf(row_sum<LPR>(dot8(x8, x8)) * (1.0f / DH) + a.eps);
      const uint64_t r2 = f2_pack(r, r);
#pragma unroll
      for (int i = 0; i < 4; ++i) x8.p[i] = f2_mul(x8.p[i], f2_mul(r2, w8.p[i]));
      x8.to(v);
      if (kRot) turn<kHalves>(v, c, s, 1.0f);
      if (h < a.heads[t]) store8<DH, kHalves>(y + h * DH, l, v);
    }
  }
}

// The gradients.  dw is summed in registers over a warp's items (a sum over
// an item's rows first, so that a long run of additions does not lose bits),
// over the block in shared memory, and over the blocks by norm_dw_kernel, all
// in a fixed order.
template <int DH, typename T, bool kHalves, bool kRot>
__global__ void __launch_bounds__(kNormThreads, 2) norm_rope_bwd_kernel(const NormArgs a, int* status) {
  constexpr int LPR = DH / 8, RPW = 32 / LPR;
  __shared__ float part[kNormWarps][2][DH];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPR, grp = lane / LPR;
  float acc[2][8] = {};
  for (Items it(a.chunks[0] + a.chunks[1]); it.n < a.N; it.next()) {
    const int t = it.chunk >= a.chunks[0];
    const int h0 = (t ? it.chunk - a.chunks[0] : it.chunk) * a.rows[t] * RPW + grp;
    const T* x = static_cast<const T*>(a.x[t]) + it.n * a.sn[t];
    const __nv_bfloat16* dy = static_cast<const __nv_bfloat16*>(a.dy[t]) + it.n * a.heads[t] * DH;
    Raw<T> raw[kRows<T>];
    Raw<__nv_bfloat16> grad[kRows<T>];
#pragma unroll
    for (int u = 0; u < kRows<T>; ++u) {
      const int h = h0 + u * RPW;
      raw[u] = Raw<T>{};
      grad[u] = Raw<__nv_bfloat16>{};
      if (u < a.rows[t] && h < a.heads[t]) {
        load8<DH, kHalves>(raw[u], x + h * a.sh[t], l);
        load8<DH, kHalves>(grad[u], dy + h * DH, l);
      }
    }
    float c[4], s[4];
    if (!angles<kRot>(a, it.n, l, c, s, status)) {
      if (a.fill) fill_nan<DH, kHalves, T>(a, it.n, t, l, h0, RPW);
      continue;
    }
    float w[8], dw[8] = {};
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = a.w[t] ? __ldg(a.w[t] + channel<DH, kHalves>(l, e)) : 1.0f;
    const Eight w8(w);
    Eight dw8(dw);
    T* dx = static_cast<T*>(a.y[t]) + it.n * a.heads[t] * DH;
#pragma unroll
    for (int u = 0; u < kRows<T>; ++u) {
      if (u >= a.rows[t]) break;
      const int h = h0 + u * RPW;
      float v[8], g[8];
      values(raw[u], v);
      values(grad[u], g);
      if (kRot) turn<kHalves>(g, c, s, -1.0f);
      Eight x8(v), g8(g);
      const float r = rsqrtf(row_sum<LPR>(dot8(x8, x8)) * (1.0f / DH) + a.eps);
      const bool live = h < a.heads[t];  // a missing row's 0 * inf (eps = 0) must not reach dw
      const uint64_t r2 = f2_pack(r, r);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x8.p[i] = f2_mul(x8.p[i], r2);
        if (live) dw8.p[i] = f2_fma(g8.p[i], x8.p[i], dw8.p[i]);
        g8.p[i] = f2_mul(g8.p[i], w8.p[i]);
      }
      const float m = row_sum<LPR>(dot8(g8, x8)) * (-1.0f / DH);
      const uint64_t m2 = f2_pack(m, m);
#pragma unroll
      for (int i = 0; i < 4; ++i) g8.p[i] = f2_mul(r2, f2_fma(x8.p[i], m2, g8.p[i]));
      g8.to(g);
      if (live) store8<DH, kHalves>(dx + h * DH, l, g);
    }
    dw8.to(dw);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      acc[0][e] += t ? 0.0f : dw[e];
      acc[1][e] += t ? dw[e] : 0.0f;
    }
  }
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float v = acc[t][e];
#pragma unroll
      for (int m = LPR; m < 32; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
      if (grp == 0) part[warp][t][channel<DH, kHalves>(l, e)] = v;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * DH; i += kNormThreads) {
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < kNormWarps; ++k) v += part[k][i / DH][i % DH];
    a.part[(int64_t)blockIdx.x * 2 * DH + i] = v;
  }
}

// dw[t][c] = sum over the blocks' partial sums, in 64 bits.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* __restrict__ part, int blocks, int DH,
                                                       float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ double sum[32][33];
  const int i = blockIdx.x * 32 + threadIdx.x;
  double v = 0.0;
#pragma unroll 10
  for (int b = threadIdx.y; b < blocks; b += 32) v += part[(int64_t)b * 2 * DH + i];
  sum[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0) {
    for (int k = 1; k < 32; ++k) v += sum[k][threadIdx.x];
    float* dw = i < DH ? dwq : dwk;
    if (dw) dw[i % DH] = (float)v;
  }
}

// table[p][j] = (cos, sin) of p * theta^(-i / n) for pair j, the i-th of its
// axis's n pairs; the angle is formed in 64 bits, where a position of 2^20
// still leaves it exact to 1e-10.
__global__ void rope_table_kernel(int P, int half, int end0, int end1, int end2, double theta,
                                  float2* __restrict__ table) {
  const int64_t k = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (k >= (int64_t)P * half) return;
  const int p = (int)(k / half), j = (int)(k - (int64_t)p * half);
  double c = 1.0, s = 0.0;
  if (j < end2) {
    const int b = j < end0 ? 0 : j < end1 ? end0 : end1;
    const int n = (j < end0 ? end0 : j < end1 ? end1 : end2) - b;
    sincos((double)p * pow(theta, -(double)(j - b) / n), &s, &c);
  }
  table[k] = make_float2((float)c, (float)s);
}

template <int DH, typename T, bool kHalves, bool kRot>
cudaError_t launch_as(const DevCtx& c, const NormArgs& a, bool backward, int* blocks) {
  const int64_t items = a.N * (a.chunks[0] + a.chunks[1]);
  int64_t grid = ceil_div(items, kNormWarps);
  const int64_t cap = (int64_t)c.num_sms * (backward ? 2 : 4);
  if (grid > cap) grid = cap;
  if (grid > kNormBlocks) grid = kNormBlocks;
  *blocks = (int)grid;
  if (grid == 0) return cudaSuccess;
  if (backward)
    norm_rope_bwd_kernel<DH, T, kHalves, kRot><<<(unsigned)grid, kNormThreads, 0, c.stream>>>(a, c.status);
  else
    norm_rope_kernel<DH, T, kHalves, kRot><<<(unsigned)grid, kNormThreads, 0, c.stream>>>(a, c.status);
  return cudaGetLastError();
}

template <int DH, typename T>
cudaError_t launch_dt(const DevCtx& c, const NormArgs& a, bool halves, bool backward, int* blocks) {
  if (a.end2 == 0) return launch_as<DH, T, false, false>(c, a, backward, blocks);
  return halves ? launch_as<DH, T, true, true>(c, a, backward, blocks)
                : launch_as<DH, T, false, true>(c, a, backward, blocks);
}

}  // namespace

cudaError_t launch_rope_table(const DevCtx& c, int P, int d_h, const int* axes, double theta, float* table) {
  const int64_t n = (int64_t)P * (d_h / 2);
  rope_table_kernel<<<(unsigned)ceil_div(n, 256), 256, 0, c.stream>>>(
      P, d_h / 2, axes[0], axes[0] + axes[1], axes[0] + axes[1] + axes[2], theta, reinterpret_cast<float2*>(table));
  return cudaGetLastError();
}

cudaError_t launch_norm_rope(const DevCtx& c, NormArgs a, int d_h, bool bf16, bool halves, bool backward,
                             float* dwq, float* dwk, int* launches) {
  // Heads are split evenly over chunks of at most kRows rows per lane group.
  const int rpw = 256 / d_h, most = bf16 ? kRows<__nv_bfloat16> : kRows<float>;
  for (int t = 0; t < 2; ++t) {
    a.chunks[t] = (int)ceil_div(a.heads[t], (int64_t)rpw * most);
    a.rows[t] = a.chunks[t] ? (int)ceil_div(a.heads[t], (int64_t)rpw * a.chunks[t]) : 0;
  }
  a.half = d_h / 2;
  int blocks = 0;
  *launches = 0;
  if (a.N > 0) {
    cudaError_t e;
    if (d_h == 128)
      e = bf16 ? launch_dt<128, __nv_bfloat16>(c, a, halves, backward, &blocks)
               : launch_dt<128, float>(c, a, halves, backward, &blocks);
    else
      e = bf16 ? launch_dt<64, __nv_bfloat16>(c, a, halves, backward, &blocks)
               : launch_dt<64, float>(c, a, halves, backward, &blocks);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  if (backward && (dwq || dwk)) {
    norm_dw_kernel<<<2 * d_h / 32, dim3(32, 32), 0, c.stream>>>(a.part, blocks, d_h, dwq, dwk);
    ++*launches;
    return cudaGetLastError();
  }
  return cudaSuccess;
}

}  // namespace moga

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
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace moga {
namespace {

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
__device__ bool segments_ok(const CrossArgs& a, int* status) {
  bool bad = false;
  for (int s = threadIdx.x; s < a.S; s += blockDim.x) {
    const Seg g = segment(a, s);
    bad |= g.q0 < 0 || g.q1 < g.q0 || g.q1 > a.N || g.k0 < 0 || g.k1 < g.k0 || g.k1 > a.L;
    if (a.kv_off) bad |= a.kv_off[s + 1] < a.kv_off[s] || a.kv_off[s + 1] > a.L;
  }
  if (!__syncthreads_or(bad)) return true;
  if (threadIdx.x == 0 && status) atomicOr(status, DEV_RANGE);
  return false;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}
template <int C>
__device__ __forceinline__ void load_row(const void* base, int64_t sn, int64_t sh, int64_t row, int h, int lane,
                                         float (&x)[C]) {
  const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(base) + row * sn + h * sh + lane * C;
#pragma unroll
  for (int i = 0; i < C; ++i) x[i] = __bfloat162float(p[i]);
}
template <int C>
__device__ __forceinline__ void store_row(void* base, int64_t at, int lane, const float (&x)[C], float f) {
  __nv_bfloat16* p = static_cast<__nv_bfloat16*>(base) + at + lane * C;
#pragma unroll
  for (int i = 0; i < C; ++i) p[i] = __float2bfloat16(x[i] * f);
}
template <int C>
__device__ __forceinline__ float dot(const float (&x)[C], const float (&y)[C]) {
  float v = 0.0f;
#pragma unroll
  for (int i = 0; i < C; ++i) v = fmaf(x[i], y[i], v);
  return warp_sum(v);
}

// One warp for each (query row, head): out and lse, or (kBwd) dq and D.
template <int DH, bool kBwd>
__global__ void __launch_bounds__(256) cross_rows_kernel(const CrossArgs a, int* status) {
  constexpr int C = DH / 32;
  if (!segments_ok(a, status)) return;
  const int lane = threadIdx.x & 31;
  const float scale = rsqrtf((float)DH);
  const int64_t nw = (int64_t)gridDim.x * 8;
  for (int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); w < a.N * a.H; w += nw) {
    const int64_t n = w / a.H;
    const int h = (int)(w - n * a.H), hk = h / (a.H / a.Hkv);
    Seg g{0, 0, 0, 0};
    for (int s = 0; s < a.S; ++s) {
      const Seg t = segment(a, s);
      if (n >= t.q0 && n < t.q1) g = t;
    }
    if (g.q1 <= g.q0) continue;  // a row of no segment
    float q[C], o[C] = {}, k[C], v[C];
    load_row<C>(a.q, a.q_sn, a.q_sh, n, h, lane, q);
    const int64_t at = (n * a.H + h) * DH;
    if (!kBwd) {
      float m = -INFINITY, l = 0.0f;
      for (int j = g.k0; j < g.k1; ++j) {
        load_row<C>(a.k, a.k_sn, a.k_sh, j, hk, lane, k);
        load_row<C>(a.v, a.v_sn, a.v_sh, j, hk, lane, v);
        const float s = dot(q, k) * scale, mn = fmaxf(m, s);
        const float f = expf(m - mn), p = expf(s - mn);
        m = mn;
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < C; ++i) o[i] = o[i] * f + p * v[i];
      }
      store_row<C>(a.out, at, lane, o, l > 0.0f ? 1.0f / l : 0.0f);
      if (a.lse && lane == 0) a.lse[(int64_t)h * a.N + n] = m + logf(l);
    } else {
      float d[C], r[C], acc[C] = {};
      load_row<C>(a.dout, (int64_t)a.H * DH, DH, n, h, lane, d);
      load_row<C>(a.out, (int64_t)a.H * DH, DH, n, h, lane, r);
      const float D = dot(d, r), lse = a.lse[(int64_t)h * a.N + n];
      for (int j = g.k0; j < g.k1; ++j) {
        load_row<C>(a.k, a.k_sn, a.k_sh, j, hk, lane, k);
        load_row<C>(a.v, a.v_sn, a.v_sh, j, hk, lane, v);
        const float ds = expf(dot(q, k) * scale - lse) * (dot(d, v) - D);
#pragma unroll
        for (int i = 0; i < C; ++i) acc[i] = fmaf(ds, k[i], acc[i]);
      }
      store_row<C>(a.dq, at, lane, acc, scale);
      if (lane == 0) a.dsum[(int64_t)h * a.N + n] = D;
    }
  }
}

// One warp for each (key row, key head): dk and dv.
template <int DH>
__global__ void __launch_bounds__(256) cross_keys_kernel(const CrossArgs a, int* status) {
  constexpr int C = DH / 32;
  if (!segments_ok(a, status)) return;
  const int lane = threadIdx.x & 31, share = a.H / a.Hkv;
  const float scale = rsqrtf((float)DH);
  const int64_t nw = (int64_t)gridDim.x * 8;
  for (int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); w < a.L * a.Hkv; w += nw) {
    const int64_t j = w / a.Hkv;
    const int hk = (int)(w - j * a.Hkv);
    Seg g{0, 0, 0, 0};
    for (int s = 0; s < a.S; ++s) {
      const Seg t = segment(a, s);
      if (j >= t.k0 && j < t.k1) g = t;
    }
    if (g.k1 <= g.k0) continue;
    float k[C], v[C], q[C], d[C], dk[C] = {}, dv[C] = {};
    load_row<C>(a.k, a.k_sn, a.k_sh, j, hk, lane, k);
    load_row<C>(a.v, a.v_sn, a.v_sh, j, hk, lane, v);
    for (int h = hk * share; h < (hk + 1) * share; ++h)
      for (int n = g.q0; n < g.q1; ++n) {
        load_row<C>(a.q, a.q_sn, a.q_sh, n, h, lane, q);
        load_row<C>(a.dout, (int64_t)a.H * DH, DH, n, h, lane, d);
        const int64_t i = (int64_t)h * a.N + n;
        const float p = expf(dot(q, k) * scale - a.lse[i]), ds = p * (dot(d, v) - a.dsum[i]);
#pragma unroll
        for (int e = 0; e < C; ++e) {
          dk[e] = fmaf(ds, q[e], dk[e]);
          dv[e] = fmaf(p, d[e], dv[e]);
        }
      }
    const int64_t at = (j * a.Hkv + hk) * DH;
    store_row<C>(a.dk, at, lane, dk, scale);
    store_row<C>(a.dv, at, lane, dv, 1.0f);
  }
}

unsigned blocks_for(const DevCtx& c, int64_t warps) {
  const int64_t b = ceil_div(warps, 8), cap = (int64_t)c.num_sms * 64;
  return (unsigned)(b < cap ? b : cap);
}

}  // namespace

size_t cross_fwd_ws_bytes(int64_t, int64_t, int, int, int, int) { return 0; }
size_t cross_bwd_ws_bytes(int64_t N, int64_t, int H, int, int, int) { return (size_t)N * H * 4; }

cudaError_t launch_cross_attn(const DevCtx& c, const CrossArgs& a, uint8_t*, int* launches) {
  *launches = 0;
  if (a.N == 0) return cudaSuccess;
  (a.d_h == 128 ? cross_rows_kernel<128, false> : cross_rows_kernel<64, false>)<<<blocks_for(c, a.N * a.H), 256, 0, c.stream>>>(a, c.status);
  *launches = 1;
  return cudaGetLastError();
}

cudaError_t launch_cross_bwd(const DevCtx& c, const CrossArgs& args, uint8_t* ws, int* launches) {
  CrossArgs a = args;
  a.dsum = reinterpret_cast<float*>(ws);
  *launches = 0;
  if (a.N > 0) {
    (a.d_h == 128 ? cross_rows_kernel<128, true> : cross_rows_kernel<64, true>)<<<blocks_for(c, a.N * a.H), 256, 0, c.stream>>>(a, c.status);
    ++*launches;
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (a.L > 0) {
    (a.d_h == 128 ? cross_keys_kernel<128> : cross_keys_kernel<64>)<<<blocks_for(c, a.L * a.Hkv), 256, 0, c.stream>>>(a, c.status);
    ++*launches;
    return cudaGetLastError();
  }
  return cudaSuccess;
}

}  // namespace moga

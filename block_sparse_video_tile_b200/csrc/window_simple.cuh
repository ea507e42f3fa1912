// window_simple.cuh -- the gradient of the window attention, one warp per
// row: the formulas as they stand, lane c holding channels c, c + 32, ...
#pragma once

#include <cmath>

#include "vsa_ptx.cuh"
#include "window_args.cuh"

namespace vsa {

template <bool F16>
__device__ __forceinline__ float elem(const uint16_t* p) {
  if (F16) return __half2float(*reinterpret_cast<const __half*>(p));
  return __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p));
}
template <bool F16>
__device__ __forceinline__ void put(uint16_t* p, float f) {
  if (F16) *reinterpret_cast<__half*>(p) = __float2half_rn(f);
  else *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(f);
}
__device__ __forceinline__ float warp_sum(float v) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int D, bool F16>
__device__ __forceinline__ void load_row(const uint16_t* p, int lane, float (&f)[D / 32]) {
  for (int c = 0; c < D / 32; ++c) f[c] = elem<F16>(p + lane + 32 * c);
}
template <int D>
__device__ __forceinline__ float dot(const float (&x)[D / 32], const float (&y)[D / 32]) {
  float s = 0.f;
  for (int c = 0; c < D / 32; ++c) s = fmaf(x[c], y[c], s);
  return warp_sum(s);
}

// One warp per (query row, head, batch): delta = dO . O and dQ.
template <int D, bool F16>
__global__ void window_dq_simple(const WinArgs a) {
  const int lane = threadIdx.x % 32, i = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
  const int h = blockIdx.y, b = blockIdx.z;
  if (i >= a.Nq) return;
  const int len = win_len(a, b);
  const RowVis vis = row_vis(a, len, win_start(a, b, len) + i);
  const uint16_t* kp = a.k + b * a.ks[0] + (h / a.group) * a.ks[2];
  const uint16_t* vp = a.v + b * a.vs[0] + (h / a.group) * a.vs[2];
  float q[D / 32], g[D / 32], x[D / 32], y[D / 32], dq[D / 32] = {};
  load_row<D, F16>(a.q + b * a.qs[0] + i * a.qs[1] + h * a.qs[2], lane, q);
  load_row<D, F16>(a.d_o + b * a.dos[0] + i * a.dos[1] + h * a.dos[2], lane, g);
  load_row<D, F16>(a.o + b * a.os[0] + i * a.os[1] + h * a.os[2], lane, x);
  const size_t r = (static_cast<size_t>(b) * a.Hq + h) * a.Nq + i;
  const float delta = dot<D>(g, x), lse2 = a.lse[r] * 1.4426950408889634f;
  if (lane == 0) a.delta[r] = delta;
  for (int j = vis.first > 0 ? 0 : vis.lo; j < vis.hi; ++j) {
    if (j == vis.first && j < vis.lo) j = vis.lo;
    if (j >= vis.hi) break;
    load_row<D, F16>(kp + j * a.ks[1], lane, x);
    load_row<D, F16>(vp + j * a.vs[1], lane, y);
    const float p = exp2f(dot<D>(q, x) * a.scale_log2 - lse2);
    const float ds = p * (dot<D>(g, y) - delta);
    for (int c = 0; c < D / 32; ++c) dq[c] = fmaf(ds, x[c], dq[c]);
  }
  uint16_t* op = a.dq + b * a.dqs[0] + i * a.dqs[1] + h * a.dqs[2];
  for (int c = 0; c < D / 32; ++c) put<F16>(op + lane + 32 * c, dq[c] * a.scale);
}

// One warp per (key row, key/value head, batch), over the queries that see
// it in order: dK and dV.
template <int D, bool F16>
__global__ void window_dkv_simple(const WinArgs a) {
  const int lane = threadIdx.x % 32, j = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
  const int hk = blockIdx.y, b = blockIdx.z;
  if (j >= a.Nk) return;
  const int len = win_len(a, b), start = win_start(a, b, len);
  float dk[D / 32] = {}, dv[D / 32] = {};
  if (j < len) {
    float k[D / 32], v[D / 32], q[D / 32], g[D / 32];
    load_row<D, F16>(a.k + b * a.ks[0] + j * a.ks[1] + hk * a.ks[2], lane, k);
    load_row<D, F16>(a.v + b * a.vs[0] + j * a.vs[1] + hk * a.vs[2], lane, v);
    const int u = j / a.unit;
    const long long p0 = 1ll * u * a.unit;
    const long long p1 = j < a.sink_tok ? (1ll << 40) : (static_cast<long long>(u) + a.window) * a.unit;
    const long long i0 = max(p0 - start, 0ll), i1 = min(p1 - start, static_cast<long long>(a.Nq));
    for (int h = hk * a.group; h < (hk + 1) * a.group; ++h) {
      for (long long i = i0; i < i1; ++i) {
        load_row<D, F16>(a.q + b * a.qs[0] + i * a.qs[1] + h * a.qs[2], lane, q);
        load_row<D, F16>(a.d_o + b * a.dos[0] + i * a.dos[1] + h * a.dos[2], lane, g);
        const size_t r = (static_cast<size_t>(b) * a.Hq + h) * a.Nq + i;
        const float p = exp2f(dot<D>(q, k) * a.scale_log2 - a.lse[r] * 1.4426950408889634f);
        const float ds = p * (dot<D>(g, v) - a.delta[r]);
        for (int c = 0; c < D / 32; ++c) {
          dv[c] = fmaf(p, g[c], dv[c]);
          dk[c] = fmaf(ds, q[c], dk[c]);
        }
      }
    }
  }
  uint16_t* kp = a.dk + b * a.dks[0] + j * a.dks[1] + hk * a.dks[2];
  uint16_t* vp = a.dv + b * a.dvs[0] + j * a.dvs[1] + hk * a.dvs[2];
  for (int c = 0; c < D / 32; ++c) {
    put<F16>(kp + lane + 32 * c, dk[c] * a.scale);
    put<F16>(vp + lane + 32 * c, dv[c]);
  }
}

}  // namespace vsa

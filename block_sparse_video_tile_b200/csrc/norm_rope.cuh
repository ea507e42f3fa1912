// norm_rope.cuh -- RMS norm of query and key heads and their position
// rotation in one pass, and the gradient.
//
// Row x of d channels (one token, one head):
//   r = 1 / sqrt(mean(x^2) + eps),  u = r x,  y = R (w * u)
// with R turning channel pair p by the angle of the token's t, y or x
// position.  R is orthogonal, so with g = R^T dy and h = g * w:
//   dw = sum over rows of g * u,   dx = r (h - u mean(h * u)).
//
// Bound by HBM: 4 bytes a channel forward (read x, write y), 6 backward (read
// x and dy, write dx), against ~8 and ~16 float operations.  So a row stays
// in registers between its one read and its one write, 16 bytes a lane: d/8
// lanes hold a row, 4 channel pairs a lane.  A lane keeps its token's four
// (cos, sin) pairs and its channels' weights for all the heads it walks
// (kRows rows of loads in flight at a time), and the table they come from
// (a few KB per axis) stays in L1 and L2: HBM sees x and y only.
#pragma once

#include <cstdint>

#include "vsa_ptx.cuh"

namespace vsa {

constexpr int kNrThreads = 256;
constexpr int kNrRows = 4;               // rows a lane loads before it computes the first

// One side; extents as in vsa_qk_side, strides in elements.
struct NrSide {
  int N, H;                  // tokens, heads
  int Hh, W;                 // rows and columns of the grid (N = T * Hh * W)
  int groups, chunks, hpc;   // token groups, head chunks, heads per chunk
  int items;                 // B * groups * chunks
  const uint16_t *x, *dy;    // dy: backward
  uint16_t* out;             // y, or dx backward
  long long xs[3], ys[3], os[3];   // (b, n, h) strides of x, dy, out
  const void* weight;
  int weight_f32;
  const float2* table;       // (cos, sin)
  int toff1, toff2;          // first table row of the y and of the x pairs
  float* partial;            // backward: [gridDim.x, D] sums of g * u of each CTA
};

struct NrArgs {
  NrSide s[2];
  int c0, c1, c2;            // channel pairs turned by t, y, x
  float eps;
};

// A lane's 8 channels as 4 pairs: interleaved: channels 8l .. 8l+7; halves:
// channels 4l .. 4l+3 and D/2 + 4l .. D/2 + 4l+3.
struct NrRaw {
  uint32_t w[4];
};

__device__ __forceinline__ uint4 ld_stream16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(reinterpret_cast<uint64_t>(p)));
  return v;
}
__device__ __forceinline__ uint2 ld_stream8(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.b32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "l"(reinterpret_cast<uint64_t>(p)));
  return v;
}

template <int D, bool IL>
__device__ __forceinline__ NrRaw nr_load(const uint16_t* row, int l) {
  NrRaw r;
  if (IL) {
    const uint4 v = ld_stream16(row + 8 * l);
    r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
  } else {
    const uint2 a = ld_stream8(row + 4 * l), b = ld_stream8(row + D / 2 + 4 * l);
    r.w[0] = a.x; r.w[1] = a.y; r.w[2] = b.x; r.w[3] = b.y;
  }
  return r;
}

template <bool F16, bool IL>
__device__ __forceinline__ void nr_unpack(const NrRaw& r, float (&a)[4], float (&b)[4]) {
  if (IL) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = unpack_elem2<F16>(r.w[e]);
      a[e] = f.x;
      b[e] = f.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float2 f = unpack_elem2<F16>(r.w[e]), g = unpack_elem2<F16>(r.w[2 + e]);
      a[2 * e] = f.x; a[2 * e + 1] = f.y;
      b[2 * e] = g.x; b[2 * e + 1] = g.y;
    }
  }
}

template <int D, bool F16, bool IL>
__device__ __forceinline__ void nr_store(uint16_t* row, int l, const float (&a)[4], const float (&b)[4]) {
  if (IL) {
    *reinterpret_cast<uint4*>(row + 8 * l) = make_uint4(pack_elem2<F16>(a[0], b[0]), pack_elem2<F16>(a[1], b[1]),
                                                        pack_elem2<F16>(a[2], b[2]), pack_elem2<F16>(a[3], b[3]));
  } else {
    *reinterpret_cast<uint2*>(row + 4 * l) = make_uint2(pack_elem2<F16>(a[0], a[1]), pack_elem2<F16>(a[2], a[3]));
    *reinterpret_cast<uint2*>(row + D / 2 + 4 * l) =
        make_uint2(pack_elem2<F16>(b[0], b[1]), pack_elem2<F16>(b[2], b[3]));
  }
}

// Sum over the LPR lanes that hold one row.
template <int LPR>
__device__ __forceinline__ float nr_row_sum(float v) {
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int D, bool F16, bool IL>
__device__ __forceinline__ void nr_weights(const NrSide& s, int l, float (&wa)[4], float (&wb)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) wa[e] = wb[e] = 1.f;
  if (s.weight == nullptr) return;
  if (s.weight_f32) {
    const float* w = static_cast<const float*>(s.weight);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int p = 4 * l + e;
      wa[e] = __ldg(w + (IL ? 2 * p : p));
      wb[e] = __ldg(w + (IL ? 2 * p + 1 : p + D / 2));
    }
  } else {
    nr_unpack<F16, IL>(nr_load<D, IL>(static_cast<const uint16_t*>(s.weight), l), wa, wb);
  }
}

// cos and sin of the lane's four pairs at token n.
template <int D>
__device__ __forceinline__ void nr_angles(const NrArgs& a, const NrSide& s, int n, int l, float2 (&cs)[4]) {
  if (s.table == nullptr) {
#pragma unroll
    for (int e = 0; e < 4; ++e) cs[e] = make_float2(1.f, 0.f);
    return;
  }
  const int yx = n / s.W, px = n - yx * s.W;
  const int pt = yx / s.Hh, py = yx - pt * s.Hh;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int p = 4 * l + e;
    long long at;
    if (p < a.c0) at = static_cast<long long>(pt) * a.c0 + p;
    else if (p < a.c0 + a.c1) at = s.toff1 + static_cast<long long>(py) * a.c1 + (p - a.c0);
    else at = s.toff2 + static_cast<long long>(px) * a.c2 + (p - a.c0 - a.c1);
    cs[e] = __ldg(s.table + at);
  }
}

// blockIdx.y is the side; a work item is (batch, token group, head chunk).
template <int D, bool F16, bool IL, bool BWD>
__global__ void __launch_bounds__(kNrThreads) norm_rope_kernel(const __grid_constant__ NrArgs a) {
  constexpr int LPR = D / 8;                       // lanes a row
  constexpr int TOK = kNrThreads / LPR;            // tokens a CTA works on at a time
  constexpr int U = BWD ? kNrRows / 2 : kNrRows;   // backward holds two tensors' rows
  const NrSide& s = a.s[blockIdx.y];
  const int l = threadIdx.x % LPR, tok = threadIdx.x / LPR;
  float wa[4], wb[4];
  nr_weights<D, F16, IL>(s, l, wa, wb);
  float da[4] = {0.f, 0.f, 0.f, 0.f}, db[4] = {0.f, 0.f, 0.f, 0.f};   // the lane's share of dweight

  for (int it = blockIdx.x; it < s.items; it += gridDim.x) {
    const int chunk = it % s.chunks, bg = it / s.chunks;
    const int grp = bg % s.groups, b = bg / s.groups;
    const int n = grp * TOK + tok;
    const bool live = n < s.N;
    const int nn = live ? n : s.N - 1;             // idle lanes read a real row and write nothing
    const int h1 = min(s.H, (chunk + 1) * s.hpc);
    const uint16_t* xr = s.x + b * s.xs[0] + nn * s.xs[1];
    const uint16_t* gr = BWD ? s.dy + b * s.ys[0] + nn * s.ys[1] : nullptr;
    uint16_t* outr = s.out + b * s.os[0] + nn * s.os[1];
    float2 cs[4];
    nr_angles<D>(a, s, nn, l, cs);
    for (int h = chunk * s.hpc; h < h1; h += U) {
      NrRaw x[U], g[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int hh = min(h + u, h1 - 1);
        x[u] = nr_load<D, IL>(xr + hh * s.xs[2], l);
        if (BWD) g[u] = nr_load<D, IL>(gr + hh * s.ys[2], l);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float xa[4], xb[4];
        nr_unpack<F16, IL>(x[u], xa, xb);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) ss = fmaf(xa[e], xa[e], fmaf(xb[e], xb[e], ss));
        const float r = rsqrtf(nr_row_sum<LPR>(ss) * (1.f / D) + a.eps);
        float ya[4], yb[4];
        if (!BWD) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float va = xa[e] * r * wa[e], vb = xb[e] * r * wb[e];
            ya[e] = va * cs[e].x - vb * cs[e].y;
            yb[e] = va * cs[e].y + vb * cs[e].x;
          }
        } else {
          float ga[4], gb[4];
          nr_unpack<F16, IL>(g[u], ga, gb);
          float hu = 0.f;
          const bool count = live && h + u < h1;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            xa[e] *= r;                            // u
            xb[e] *= r;
            const float ta = ga[e] * cs[e].x + gb[e] * cs[e].y, tb = gb[e] * cs[e].x - ga[e] * cs[e].y;
            if (count) {
              da[e] = fmaf(ta, xa[e], da[e]);
              db[e] = fmaf(tb, xb[e], db[e]);
            }
            ga[e] = ta * wa[e];                    // h
            gb[e] = tb * wb[e];
            hu = fmaf(ga[e], xa[e], fmaf(gb[e], xb[e], hu));
          }
          const float m = nr_row_sum<LPR>(hu) * (1.f / D);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ya[e] = r * (ga[e] - xa[e] * m);
            yb[e] = r * (gb[e] - xb[e] * m);
          }
        }
        if (live && h + u < h1) nr_store<D, F16, IL>(outr + (h + u) * s.os[2], l, ya, yb);
      }
    }
  }

  if (BWD && s.partial != nullptr) {
    // the CTA's sum of g * u: over the warp's rows, then over the warps in order
    __shared__ float sums[kNrThreads / 32][D];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) {
        da[e] += __shfl_xor_sync(0xffffffffu, da[e], o);
        db[e] += __shfl_xor_sync(0xffffffffu, db[e], o);
      }
    }
    if (threadIdx.x % 32 < LPR) {
      float* row = sums[threadIdx.x / 32];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int p = 4 * l + e;
        row[IL ? 2 * p : p] = da[e];
        row[IL ? 2 * p + 1 : p + D / 2] = db[e];
      }
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < kNrThreads / 32; ++w) t += sums[w][threadIdx.x];
      s.partial[static_cast<size_t>(blockIdx.x) * D + threadIdx.x] = t;
    }
  }
}

// dweight[c] = sum of the CTAs' partial sums, in a fixed order: 1024 / D rows
// of threads take every (1024 / D)-th partial, then are added in order.
template <int D>
__global__ void __launch_bounds__(1024) norm_rope_dweight_kernel(const float* p0, float* dw0, const float* p1, float* dw1,
                                                                 int parts) {
  constexpr int R = 1024 / D;
  __shared__ float sums[R][D];
  const float* p = blockIdx.x == 0 ? p0 : p1;
  float* dw = blockIdx.x == 0 ? dw0 : dw1;
  if (dw == nullptr) return;
  const int c = threadIdx.x % D, r = threadIdx.x / D;
  float t = 0.f;
#pragma unroll 8
  for (int i = r; i < parts; i += R) t += p[static_cast<size_t>(i) * D + c];
  sums[r][c] = t;
  __syncthreads();
  if (r == 0) {
#pragma unroll
    for (int i = 1; i < R; ++i) t += sums[i][c];
    dw[c] = t;
  }
}

}  // namespace vsa

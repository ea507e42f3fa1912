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
// x and dy, write dx), against ~8 and ~16 float operations; close behind it
// the backward's instruction issue.  So a row stays in registers between its
// one read and its one write; d/16 lanes hold a row, 8 channel pairs a lane in
// two 16-byte pieces (fewer lanes a row: fewer shuffles for its sums); sums
// and products run on packed float32 pairs; and the backward's two sums,
// x^2 and h x, are made before r is known, so that a row has one round of
// shuffles.  A lane keeps its token's (cos, sin) and its channels' weights
// for all the heads it walks; the table they come from (a few KB per axis)
// stays in L1 and L2.
#pragma once

#include <cstdint>

#include "vsa_ptx.cuh"

namespace vsa {

constexpr int kNrThreads = 256;
constexpr int kNrRows = 2;               // heads a step: rows that a lane computes side by side
constexpr int kNrChunk = 4;              // heads that a CTA walks at least when the heads of a token are split
// Steps in a lane's ring.  Measured at the (31, 22, 40) grid with 24 heads of
// 128: forward 2 / 3 / 4 steps 118 / 112.6 / 112.9 us (5.95 TB/s, 91 % of the
// measured copy rate); backward 2 / 3 steps 163 / 188 us (6.17 TB/s, 94 %).
template <bool BWD>
__host__ __device__ constexpr int nr_stages() { return BWD ? 2 : 3; }

// One side; extents as in vsa_qk_side, strides in elements.
struct NrSide {
  int N, H;                  // tokens, heads
  int Hh, W;                 // rows and columns of the grid (N = T * Hh * W)
  int across;                // a warp's rows at a time: 0 of as many tokens, 1 of one token's heads
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

// A lane's 16 channels as 8 pairs.  Interleaved: channels 8l .. 8l+7 and
// D/2 + 8l .. D/2 + 8l+7, pairs 4l .. 4l+3 and D/4 + 4l .. D/4 + 4l+3.  Halves:
// the same channels, pairs 8l .. 8l+7.
struct NrRaw {
  uint4 v[2];
};

__device__ __forceinline__ uint4 ld_stream16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(reinterpret_cast<uint64_t>(p)));
  return v;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_dup(float x) { return f2_pack(x, x); }

template <bool IL>
__device__ __forceinline__ int nr_pair(int D, int l, int e) {
  return IL ? (e < 4 ? 4 * l + e : D / 4 + 4 * l + e - 4) : 8 * l + e;
}

template <int D>
__device__ __forceinline__ NrRaw nr_load(const uint16_t* row, int l) {
  NrRaw r;
  r.v[0] = ld_stream16(row + 8 * l);
  r.v[1] = ld_stream16(row + D / 2 + 8 * l);
  return r;
}

// First and second members of the lane's pairs, packed two by two.
template <bool F16, bool IL>
__device__ __forceinline__ void nr_unpack(const NrRaw& r, uint64_t (&a)[4], uint64_t (&b)[4]) {
  const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (IL) {
      const float2 f = unpack_elem2<F16>(w[2 * e]), g = unpack_elem2<F16>(w[2 * e + 1]);
      a[e] = f2_pack(f.x, g.x);
      b[e] = f2_pack(f.y, g.y);
    } else {
      const float2 f = unpack_elem2<F16>(w[e]), g = unpack_elem2<F16>(w[4 + e]);
      a[e] = f2_pack(f.x, f.y);
      b[e] = f2_pack(g.x, g.y);
    }
  }
}

template <int D, bool F16, bool IL>
__device__ __forceinline__ void nr_store(uint16_t* row, int l, const uint64_t (&a)[4], const uint64_t (&b)[4]) {
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float a0, a1, b0, b1;
    f2_unpack(a[e], a0, a1);
    f2_unpack(b[e], b0, b1);
    if (IL) {
      w[2 * e] = pack_elem2<F16>(a0, b0);
      w[2 * e + 1] = pack_elem2<F16>(a1, b1);
    } else {
      w[e] = pack_elem2<F16>(a0, a1);
      w[4 + e] = pack_elem2<F16>(b0, b1);
    }
  }
  *reinterpret_cast<uint4*>(row + 8 * l) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(row + D / 2 + 8 * l) = make_uint4(w[4], w[5], w[6], w[7]);
}

// Sum over the LPR lanes that hold one row.
template <int LPR>
__device__ __forceinline__ float nr_row_sum(float v) {
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float f2_sum(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return a + b;
}

template <int D, bool F16, bool IL>
__device__ __forceinline__ void nr_weights(const NrSide& s, int l, uint64_t (&wa)[4], uint64_t (&wb)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) wa[e] = wb[e] = f2_dup(1.f);
  if (s.weight == nullptr) return;
  if (s.weight_f32) {
    const float* w = static_cast<const float*>(s.weight);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int p = nr_pair<IL>(D, l, 2 * e), p1 = nr_pair<IL>(D, l, 2 * e + 1);
      wa[e] = f2_pack(__ldg(w + (IL ? 2 * p : p)), __ldg(w + (IL ? 2 * p1 : p1)));
      wb[e] = f2_pack(__ldg(w + (IL ? 2 * p + 1 : p + D / 2)), __ldg(w + (IL ? 2 * p1 + 1 : p1 + D / 2)));
    }
  } else {
    nr_unpack<F16, IL>(nr_load<D>(static_cast<const uint16_t*>(s.weight), l), wa, wb);
  }
}

// cos and sin of the lane's pairs at token n.
template <int D, bool IL>
__device__ __forceinline__ void nr_angles(const NrArgs& a, const NrSide& s, int n, int l, uint64_t (&co)[4],
                                          uint64_t (&si)[4]) {
  if (s.table == nullptr) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      co[e] = f2_dup(1.f);
      si[e] = f2_dup(0.f);
    }
    return;
  }
  const int yx = n / s.W, px = n - yx * s.W;
  const int pt = yx / s.Hh, py = yx - pt * s.Hh;
  float2 cs[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int p = nr_pair<IL>(D, l, e);
    long long at;
    if (p < a.c0) at = static_cast<long long>(pt) * a.c0 + p;
    else if (p < a.c0 + a.c1) at = s.toff1 + static_cast<long long>(py) * a.c1 + (p - a.c0);
    else at = s.toff2 + static_cast<long long>(px) * a.c2 + (p - a.c0 - a.c1);
    cs[e] = __ldg(s.table + at);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    co[e] = f2_pack(cs[2 * e].x, cs[2 * e + 1].x);
    si[e] = f2_pack(cs[2 * e].y, cs[2 * e + 1].y);
  }
}

__device__ __forceinline__ uint64_t f2_neg(uint64_t v) { return v ^ 0x8000000080000000ull; }

// blockIdx.y is the side; a work item is (batch, token group, head chunk).
// Which rows a lane group takes: of token grp * tokens + tok, heads h0 + u * hs.
// Rows that lie next to each other in memory are read by lanes next to each
// other: with the heads of a token innermost, a warp takes several heads of one
// token, else one head of several tokens (norm_rope_wan5b, [B, N, 3, H, d]
// views: 128 us when a warp took several tokens there).
template <int D>
struct NrPlace {
  int tokens, tok, h0, hs;
  __device__ __forceinline__ NrPlace(const NrSide& s) {
    constexpr int G = 512 / D;                     // lane groups a warp
    const int grp = threadIdx.x % 32 / (D / 16), warp = threadIdx.x / 32;
    tokens = s.across ? kNrThreads / 32 : kNrThreads / 32 * G;
    tok = s.across ? warp : warp * G + grp;
    h0 = s.across ? grp : 0;
    hs = s.across ? G : 1;
  }
};

// The (item, head) sequence of a lane's rows, kNrRows heads a step.  Every lane copies
// (cp.async) exactly the 16-byte pieces that it reads later, nr_stages() - 1 steps
// ahead and across items, so its ring needs no barrier and the loads in flight
// do not depend on how many registers the arithmetic takes.
template <int D, bool BWD>
struct NrLoads {
  int it, h, h1;
  const uint16_t *xr, *gr;

  __device__ __forceinline__ void start(const NrSide& s, const NrPlace<D>& at, int item, int l) {
    it = item;
    if (it >= s.items) return;
    const int chunk = it % s.chunks, bg = it / s.chunks;
    const int grp = bg % s.groups, b = bg / s.groups;
    const int nn = min(grp * at.tokens + at.tok, s.N - 1);
    h = chunk * s.hpc;
    h1 = min(s.H, h + s.hpc);
    xr = s.x + b * s.xs[0] + nn * s.xs[1] + 8 * l;
    if (BWD) gr = s.dy + b * s.ys[0] + nn * s.ys[1] + 8 * l;
  }
  // Copies the next step's rows to `dst` (this thread's place in a stage).
  __device__ __forceinline__ void step(const NrSide& s, const NrPlace<D>& at, uint32_t dst, int l) {
    if (it < s.items) {
#pragma unroll
      for (int u = 0; u < kNrRows; ++u) {
        const int hh = min(h + u * at.hs + at.h0, h1 - 1);
        const uint32_t d = dst + u * (BWD ? 4 : 2) * kNrThreads * 16;
        const uint16_t* x = xr + hh * s.xs[2];
        cp_async16(d, x, 16u);
        cp_async16(d + kNrThreads * 16, x + D / 2, 16u);
        if (BWD) {
          const uint16_t* g = gr + hh * s.ys[2];
          cp_async16(d + 2 * kNrThreads * 16, g, 16u);
          cp_async16(d + 3 * kNrThreads * 16, g + D / 2, 16u);
        }
      }
      h += kNrRows * at.hs;
      if (h >= h1) start(s, at, it + gridDim.x, l);
    }
    cp_async_commit();
  }
};

template <bool BWD>
__host__ __device__ constexpr int nr_smem_bytes() {
  return nr_stages<BWD>() * kNrRows * (BWD ? 4 : 2) * kNrThreads * 16;
}

// blockIdx.y is the side; a work item is (batch, token group, head chunk).
template <int D, bool F16, bool IL, bool BWD>
__global__ void __launch_bounds__(kNrThreads, 2) norm_rope_kernel(const __grid_constant__ NrArgs a) {
  constexpr int LPR = D / 16;                      // lanes a row
  constexpr int U = kNrRows, S = nr_stages<BWD>();
  constexpr uint32_t kPiece = kNrThreads * 16, kStage = U * (BWD ? 4 : 2) * kPiece;
  extern __shared__ __align__(128) unsigned char ring_mem[];
  const NrSide& s = a.s[blockIdx.y];
  const int l = threadIdx.x % LPR;
  const NrPlace<D> at(s);
  const uint32_t ring = smem_u32(ring_mem) + threadIdx.x * 16;
  NrLoads<D, BWD> ld;
  ld.start(s, at, blockIdx.x, l);
#pragma unroll
  for (int i = 0; i < S - 1; ++i) ld.step(s, at, ring + i * kStage, l);
  uint64_t wa[4], wb[4];
  nr_weights<D, F16, IL>(s, l, wa, wb);
  uint64_t da[4] = {0, 0, 0, 0}, db[4] = {0, 0, 0, 0};   // the lane's share of dweight
  int st = 0;

  for (int it = blockIdx.x; it < s.items; it += gridDim.x) {
    const int chunk = it % s.chunks, bg = it / s.chunks;
    const int grp = bg % s.groups, b = bg / s.groups;
    const int n = grp * at.tokens + at.tok;
    const bool live = n < s.N;
    const int nn = live ? n : s.N - 1;             // idle lanes read a real row and write nothing
    const int h1 = min(s.H, (chunk + 1) * s.hpc);
    uint16_t* outr = s.out + b * s.os[0] + nn * s.os[1];
    uint64_t co[4], si[4];
    nr_angles<D, IL>(a, s, nn, l, co, si);
    for (int h = chunk * s.hpc; h < h1; h += U * at.hs) {
      cp_async_wait<S - 2>();
      NrRaw x[U], g[U];
      const unsigned char* mine = ring_mem + threadIdx.x * 16 + st * kStage;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const unsigned char* p = mine + u * (BWD ? 4 : 2) * kPiece;
        x[u].v[0] = *reinterpret_cast<const uint4*>(p);
        x[u].v[1] = *reinterpret_cast<const uint4*>(p + kPiece);
        if (BWD) {
          g[u].v[0] = *reinterpret_cast<const uint4*>(p + 2 * kPiece);
          g[u].v[1] = *reinterpret_cast<const uint4*>(p + 3 * kPiece);
        }
      }
      ld.step(s, at, ring + (st == 0 ? S - 1 : st - 1) * kStage, l);   // the stage read in the step before
      if (++st == S) st = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint64_t xa[4], xb[4], ya[4], yb[4];
        nr_unpack<F16, IL>(x[u], xa, xb);
        uint64_t s0 = f2_mul(xa[0], xa[0]), s1 = f2_mul(xb[0], xb[0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) {
          s0 = f2_fma(xa[e], xa[e], s0);
          s1 = f2_fma(xb[e], xb[e], s1);
        }
        float ss = f2_sum(f2_add(s0, s1));
        const int hh = h + u * at.hs + at.h0;
        const bool live_row = live && hh < h1;
        if (!BWD) {
          const uint64_t r2 = f2_dup(rsqrtf(nr_row_sum<LPR>(ss) * (1.f / D) + a.eps));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint64_t va = f2_mul(f2_mul(xa[e], r2), wa[e]), vb = f2_mul(f2_mul(xb[e], r2), wb[e]);
            ya[e] = f2_fma(va, co[e], f2_neg(f2_mul(vb, si[e])));
            yb[e] = f2_fma(va, si[e], f2_mul(vb, co[e]));
          }
        } else {
          uint64_t ga[4], gb[4], tx[4], ty[4];
          nr_unpack<F16, IL>(g[u], ga, gb);
          uint64_t p0 = 0, p1 = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint64_t ta = f2_fma(ga[e], co[e], f2_mul(gb[e], si[e]));            // g = R^T dy
            const uint64_t tb = f2_fma(gb[e], co[e], f2_neg(f2_mul(ga[e], si[e])));
            tx[e] = f2_mul(ta, xa[e]);                                                 // g x
            ty[e] = f2_mul(tb, xb[e]);
            p0 = f2_fma(tx[e], wa[e], p0);                                             // h x
            p1 = f2_fma(ty[e], wb[e], p1);
            ga[e] = f2_mul(ta, wa[e]);                                                 // h
            gb[e] = f2_mul(tb, wb[e]);
          }
          float hx = f2_sum(f2_add(p0, p1));
#pragma unroll
          for (int o = 1; o < LPR; o <<= 1) {
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
            hx += __shfl_xor_sync(0xffffffffu, hx, o);
          }
          const float r = rsqrtf(ss * (1.f / D) + a.eps);
          const uint64_t rc = f2_dup(live_row ? r : 0.f), r2 = f2_dup(r);
          // dx = r h - x k, k = r^3 mean(h x): r is brought against hx first, since
          // r^3 alone leaves float32 for rows below 1e-13 or above 1e13
          const uint64_t k2 = f2_dup(-(r * hx * (1.f / D)) * r * r);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            da[e] = f2_fma(tx[e], rc, da[e]);
            db[e] = f2_fma(ty[e], rc, db[e]);
            ya[e] = f2_fma(xa[e], k2, f2_mul(ga[e], r2));
            yb[e] = f2_fma(xb[e], k2, f2_mul(gb[e], r2));
          }
        }
        if (live_row) nr_store<D, F16, IL>(outr + hh * s.os[2], l, ya, yb);
      }
    }
  }

  if (BWD && s.partial != nullptr) {
    // the CTA's sum of g * u: over the warp's rows, then over the warps in order
    __shared__ float sums[kNrThreads / 32][D];
    float fa[8], fb[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f2_unpack(da[e], fa[2 * e], fa[2 * e + 1]);
      f2_unpack(db[e], fb[2 * e], fb[2 * e + 1]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) {
        fa[e] += __shfl_xor_sync(0xffffffffu, fa[e], o);
        fb[e] += __shfl_xor_sync(0xffffffffu, fb[e], o);
      }
    }
    if (threadIdx.x % 32 < LPR) {
      float* row = sums[threadIdx.x / 32];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int p = nr_pair<IL>(D, l, e);
        row[IL ? 2 * p : p] = fa[e];
        row[IL ? 2 * p + 1 : p + D / 2] = fb[e];
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

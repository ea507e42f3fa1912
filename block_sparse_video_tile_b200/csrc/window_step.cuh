// window_step.cuh -- window attention of a few query rows against a long
// cache (single new tokens, speculative tokens).
//
// Bound by HBM: every visible K and V row is read once for each tile of 16
// query rows of its key/value head (2 * 2 * d bytes a key against 4 d flops a
// row: 16 rows are still far below the balance of the legacy tensor path, and
// the 128 rows of a tcgen05 tile would be nearly all padding).  So the rows --
// the group's heads of each query token -- fill m16 tiles of mma.sync (one
// for the usual call; further tiles read the keys again, from L2 where they
// fit), and the work is split over the keys: splits (CTAs) take contiguous runs of
// 16-key tiles, their four warps every fourth tile of the run.  A warp keeps
// its own running maximum, sum and O and its own ring of kWsStages tiles
// filled by cp.async (8 KB of K and V a tile at d = 128), so no warp waits for
// another before the end, where the four are joined through shared memory.  Up
// to kWsCluster splits are a cluster, whose CTAs then join their results through
// distributed shared memory (no second launch: window_step_small 9.0 us of two
// kernels); more go through window_combine_kernel.
#pragma once

#include "window_args.cuh"
#include "window_fwd.cuh"
#include "window_ptx.cuh"

namespace vsa {

constexpr int kWsWarps = 4, kWsThreads = 32 * kWsWarps;
constexpr int kWsKeys = 16;              // keys a tile
constexpr int kWsRows = 16;              // query rows a CTA (token-major, then head of the group)
constexpr int kWsStages = 3;
constexpr int kWsCluster = 8;            // splits that are joined as one cluster
constexpr float kWsUp = 15.f;            // fp16: P and l carry 2^kWsUp (P <= 1; why: see window_fwd.cuh)

template <int D>
struct WsSmem {
  static constexpr int kTile = 2 * kWsKeys * D * 2;              // K, then V
  static constexpr int kRing = kWsWarps * kWsStages * kTile;
  static constexpr int kJoin = kWsWarps * kWsRows * (D + 2) * 4;  // O, m, l of each warp (over the ring)
  static constexpr int kRes = (kJoin + 127) & ~127;               // the CTA's O, m, l for its cluster
  static constexpr int kEnd = kRes + kWsRows * (D + 2) * 4;
  static constexpr int kTotal = kRing > kEnd ? kRing : kEnd;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of a shared-memory location in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// grid (splits, Hkv * row tiles, B); CLUSTER: the splits of a row tile are one
// cluster.  That and splits == 1 write O and LSE, else the partial results of
// window_fwd_kernel's splits.
template <int D, bool F16, bool CLUSTER>
__global__ void __launch_bounds__(kWsThreads) window_step_kernel(const __grid_constant__ WinArgs a, int splits, float* part) {
  using L = WsSmem<D>;
  constexpr int CH = D / 8;                                       // 16-byte chunks of a row
  extern __shared__ __align__(128) unsigned char smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int split = blockIdx.x, hk = blockIdx.y % a.Hkv, r0 = (blockIdx.y / a.Hkv) * kWsRows, b = blockIdx.z;
  const int R = a.Nq * a.group;
  const int len = win_len(a, b), start = win_start(a, b, len);

  // rows of this lane in the m16 tile: lane / 4 and lane / 4 + 8
  RowVis vis[2];
  const uint16_t* qrow[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = r0 + lane / 4 + 8 * u;
    vis[u] = RowVis{0, 0, 0};
    qrow[u] = nullptr;
    if (r < R) {
      const int i = r / a.group, h = hk * a.group + r % a.group;
      vis[u] = row_vis(a, len, start + i);
      if (vis[u].hi > 0) qrow[u] = a.q + b * a.qs[0] + i * a.qs[1] + h * a.qs[2];
    }
  }
  // keys that some row of the tile sees: [0, first) and [lo, hi)
  const WinBlocks wb = win_blocks(a, len, start, r0 / a.group, min(r0 + kWsRows, R) == R ? a.Nq - 1 : (r0 + kWsRows - 1) / a.group);
  const int t_lo = wb.lo / kWsKeys;
  const int t_first = wb.hi > wb.lo ? min((wb.first + kWsKeys - 1) / kWsKeys, t_lo) : (wb.first + kWsKeys - 1) / kWsKeys;
  const int t_all = t_first + (wb.hi > wb.lo ? (wb.hi + kWsKeys - 1) / kWsKeys - t_lo : 0);
  const int t0 = static_cast<int>(static_cast<long long>(t_all) * split / splits) + warp;
  const int t1 = static_cast<int>(static_cast<long long>(t_all) * (split + 1) / splits);
  const int n = t1 > t0 ? (t1 - t0 + kWsWarps - 1) / kWsWarps : 0;   // this warp's tiles
  auto key_of = [&](int j) {
    const int t = t0 + j * kWsWarps;
    return (t < t_first ? t : t_lo + t - t_first) * kWsKeys;
  };

  const uint32_t ring = smem_u32(smem) + warp * kWsStages * L::kTile;
  const uint16_t* kp = a.k + b * a.ks[0] + hk * a.ks[2];
  const uint16_t* vp = a.v + b * a.vs[0] + hk * a.vs[2];
  // 16-byte chunk c of row r sits at chunk c ^ (r % 8) of the row (bank-free ldmatrix)
  auto load = [&](int j) {
    if (j < n) {
      const int c0 = key_of(j);
      const uint32_t dst = ring + (j % kWsStages) * L::kTile;
#pragma unroll
      for (int e = 0; e < kWsKeys * CH / 32; ++e) {
        const int at = e * 32 + lane, r = at / CH, c = at % CH, key = c0 + r;
        const bool seen = key < wb.first || (key >= wb.lo && key < wb.hi);
        const int from = seen ? key : 0;                          // (nothing is read for a key that nobody sees)
        const uint32_t d = dst + r * (D * 2) + ((c ^ (r & 7)) * 16);
        cp_async16(d, kp + from * a.ks[1] + c * 8, seen ? 16u : 0u);
        cp_async16(d + kWsKeys * D * 2, vp + from * a.vs[1] + c * 8, seen ? 16u : 0u);
      }
    }
    cp_async_commit();
  };
  for (int j = 0; j < kWsStages - 1; ++j) load(j);

  uint32_t q[D / 16][4];
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint16_t* p = qrow[e & 1];
      q[kk][e] = p == nullptr ? 0u : *reinterpret_cast<const uint32_t*>(p + 16 * kk + 8 * (e >> 1) + 2 * (lane % 4));
    }

  constexpr float kUp = F16 ? kWsUp : 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float o[D / 8][4];
#pragma unroll
  for (int t = 0; t < D / 8; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[t][e] = 0.f;

  for (int j = 0; j < n; ++j) {
    load(j + kWsStages - 1);
    cp_async_wait<kWsStages - 1>();
    __syncwarp();
    const uint32_t kt = ring + (j % kWsStages) * L::kTile, vt = kt + kWsKeys * D * 2;
    float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      // matrices: keys 0-7 and 8-15, channels 16 kk and 16 kk + 8
      uint32_t kf[4];
      const int r = (lane & 7) + ((lane >> 4) << 3), c = 2 * kk + ((lane >> 3) & 1);
      ldsm4(kt + r * (D * 2) + ((c ^ (r & 7)) * 16), kf);
      mma_16816<F16>(s[0], q[kk], kf[0], kf[1]);
      mma_16816<F16>(s[1], q[kk], kf[2], kf[3]);
    }
    // s[t][e]: key c0 + 8 t + 2 (lane % 4) + (e & 1), row u = e >> 1
    const int c0 = key_of(j);
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = c0 + 8 * t + 2 * (lane % 4) + (e & 1);
        s[t][e] = vis[e >> 1].sees(key) ? s[t][e] * a.scale_log2 : -INFINITY;
        mx[e >> 1] = fmaxf(mx[e >> 1], s[t][e]);
      }
    uint32_t p[4];
    float f[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 1));
      mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 2));
      const float mn = fmaxf(m[u], mx[u]), mu = mn == -INFINITY ? 0.f : mn;
      f[u] = ex2_approx(m[u] - mu);                               // (m = -inf: 0)
      m[u] = mn;
      float sum = 0.f;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float p0 = ex2_approx(s[t][2 * u] + (kUp - mu)), p1 = ex2_approx(s[t][2 * u + 1] + (kUp - mu));
        sum += p0 + p1;
        p[2 * t + u] = pack_elem2<F16>(p0, p1);                   // A fragment: rows u, keys 8 t ..
      }
      l[u] = l[u] * f[u] + sum;
    }
    if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
      for (int t = 0; t < D / 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][e] *= f[e >> 1];
    }
#pragma unroll
    for (int t = 0; t < D / 16; ++t) {
      // matrices: keys 0-7 and 8-15 of channels 16 t, then of 16 t + 8
      uint32_t vf[4];
      const int r = lane & 15, c = 2 * t + (lane >> 4);
      ldsm4_t(vt + r * (D * 2) + ((c ^ (r & 7)) * 16), vf);
      mma_16816<F16>(o[2 * t], p, vf[0], vf[1]);
      mma_16816<F16>(o[2 * t + 1], p, vf[2], vf[3]);
    }
    __syncwarp();                                                 // the stage may be refilled
  }

  // ---- join the four warps: O, m and l of each through shared memory
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
    l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
  }
  cp_async_wait<0>();
  __syncthreads();
  float* jo = reinterpret_cast<float*>(smem);                     // [warp][row][D]
  float* jm = jo + kWsWarps * kWsRows * D;                        // [warp][row][2]
#pragma unroll
  for (int t = 0; t < D / 8; ++t)
#pragma unroll
    for (int u = 0; u < 2; ++u)
      *reinterpret_cast<float2*>(jo + (warp * kWsRows + lane / 4 + 8 * u) * D + 8 * t + 2 * (lane % 4)) =
          make_float2(o[t][2 * u], o[t][2 * u + 1]);
  if (lane % 4 == 0) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      jm[(warp * kWsRows + lane / 4 + 8 * u) * 2] = m[u];
      jm[(warp * kWsRows + lane / 4 + 8 * u) * 2 + 1] = l[u];
    }
  }
  __syncthreads();
  constexpr int TPR = kWsThreads / kWsRows;                       // threads a row
  constexpr int CPT = D / TPR / 4;                                // float4 a thread
  const int rr = threadIdx.x / TPR, part_c = threadIdx.x % TPR, r = r0 + rr;
  float mt = -INFINITY, lt = 0.f;
  float4 acc[CPT];
  {
    float w[kWsWarps];
#pragma unroll
    for (int k = 0; k < kWsWarps; ++k) mt = fmaxf(mt, jm[(k * kWsRows + rr) * 2]);
#pragma unroll
    for (int k = 0; k < kWsWarps; ++k) {
      w[k] = mt == -INFINITY ? 0.f : ex2_approx(jm[(k * kWsRows + rr) * 2] - mt);
      lt = fmaf(w[k], jm[(k * kWsRows + rr) * 2 + 1], lt);
    }
#pragma unroll
    for (int e = 0; e < CPT; ++e) {
      acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kWsWarps; ++k) {
        const float4 x = *reinterpret_cast<const float4*>(jo + (k * kWsRows + rr) * D + 4 * (part_c + TPR * e));
        acc[e].x = fmaf(w[k], x.x, acc[e].x);
        acc[e].y = fmaf(w[k], x.y, acc[e].y);
        acc[e].z = fmaf(w[k], x.z, acc[e].z);
        acc[e].w = fmaf(w[k], x.w, acc[e].w);
      }
    }
  }
  bool write = r < R;
  if (CLUSTER) {
    // every CTA shows its rows; row rr is joined and written by CTA rr % splits
    float* res = reinterpret_cast<float*>(smem + L::kRes);        // [row][D], then [row][2]
#pragma unroll
    for (int e = 0; e < CPT; ++e) *reinterpret_cast<float4*>(res + rr * D + 4 * (part_c + TPR * e)) = acc[e];
    if (part_c == 0) *reinterpret_cast<float2*>(res + kWsRows * D + 2 * rr) = make_float2(mt, lt);
    cluster_sync();
    write = write && rr % splits == split;
    if (write) {
      const uint32_t mine = smem_u32(res);
      float ms[kWsCluster], mx = -INFINITY;
#pragma unroll
      for (int k = 0; k < kWsCluster; ++k) {
        ms[k] = -INFINITY;
        if (k < splits) ms[k] = ld_cluster2(cluster_addr(mine + (kWsRows * D + 2 * rr) * 4, k)).x;
        mx = fmaxf(mx, ms[k]);
      }
      mt = mx;
      lt = 0.f;
#pragma unroll
      for (int e = 0; e < CPT; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kWsCluster; ++k) {
        if (k >= splits) break;
        const float w = mx == -INFINITY ? 0.f : ex2_approx(ms[k] - mx);
        lt = fmaf(w, ld_cluster2(cluster_addr(mine + (kWsRows * D + 2 * rr) * 4, k)).y, lt);
#pragma unroll
        for (int e = 0; e < CPT; ++e) {
          const float4 x = ld_cluster4(cluster_addr(mine + (rr * D + 4 * (part_c + TPR * e)) * 4, k));
          acc[e].x = fmaf(w, x.x, acc[e].x);
          acc[e].y = fmaf(w, x.y, acc[e].y);
          acc[e].z = fmaf(w, x.z, acc[e].z);
          acc[e].w = fmaf(w, x.w, acc[e].w);
        }
      }
    }
    cluster_sync();                                               // nobody leaves while its rows are read
  }
  if (!write) return;
  // (lt = 0: the row sees nothing; a NaN among what it sees stays one)
  const float inv = lt == 0.f ? 0.f : 1.f / lt;
  const float lse = lt == 0.f ? -INFINITY : (mt - kUp + log2f(lt)) * 0.69314718055994530942f;
  const int i = r / a.group, h = hk * a.group + r % a.group;
  const size_t row = (static_cast<size_t>(b) * a.Hq + h) * a.Nq + i, rows = static_cast<size_t>(a.B) * a.Hq * a.Nq;
  const bool partial = !CLUSTER && splits > 1;
  uint16_t* out = a.out + b * a.os[0] + i * a.os[1] + h * a.os[2];
  float* po = partial ? part + (split * rows + row) * D : nullptr;
#pragma unroll
  for (int e = 0; e < CPT; ++e) {
    const int ch = 4 * (part_c + TPR * e);
    const float4 x = make_float4(acc[e].x * inv, acc[e].y * inv, acc[e].z * inv, acc[e].w * inv);
    if (partial) *reinterpret_cast<float4*>(po + ch) = x;
    else *reinterpret_cast<uint2*>(out + ch) = make_uint2(pack_elem2<F16>(x.x, x.y), pack_elem2<F16>(x.z, x.w));
  }
  if (part_c == 0) {
    if (partial) part[splits * rows * D + split * rows + row] = lse;
    else a.lse[row] = lse;
  }
}

}  // namespace vsa

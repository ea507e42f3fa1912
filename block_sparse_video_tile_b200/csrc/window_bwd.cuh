// window_bwd.cuh -- gradient of the window attention for sm_100a, from the
// forward's O and LSE:
//   P = exp(scale Q K^T - LSE),  dP = dO V^T,  delta = rowsum(dO * O),
//   dS = P * (dP - delta),  dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO
//
// Two kernels, so that no sum is made by atomics and every result has the
// same bits each time: window_dq_kernel walks the keys of 128 query rows
// (three products a block: S, dP, dQ; it also writes delta), and
// window_dkv_kernel walks the queries of 128 key rows, over all query heads
// of the key/value head (four products: S^T, dP^T, dV, dK).  S and dP are
// made twice: 7 products of 128 x 128 x d a block pair where 5 would do, in
// exchange for no float32 dQ in memory (128 KB of atomic traffic a pair).
//
// Both are bound by the tensor pipe (1536 and 2048 clk a block at d = 128)
// with the exponential unit (1024 clk) next.  The elementwise warps work on
// the block in two halves of 64 columns (a warpgroup each, thread = row), and
// write their 16-bit operand over the scores it came from, so P and dS never
// leave TMEM.  Measured (window_bwd_wan5b, 6 heads): dQ 674-690 us, dK/dV
// 1013-1020 us in bursts, tensor pipe 68-70 % active.  Not taken: 1/8 to 3/8 of
// the exponentials on the FMA pipe 0 to 5 % slower; P^T released in three parts
// 0.6 % faster, not worth its code; a warp of its own for dV's first part 3 %
// slower.
//
// Rounding: P and dS are rounded to the 16-bit type as MMA operands; scores,
// dP, delta and the accumulators are float32; results are rounded once.
//
// fp16 holds 2^-14 .. 2^16 in full precision, and P is about one over the
// number of keys, dS smaller still by dO: unscaled, 4480 keys left dQ with 0.6 %
// of error for dO of 1e-3 and 5.7 % for 1e-4 (0.03 % now), and dO of 1e4 with
// infinities.  So the fp16 kernels carry P times 2^12 (P <= 1), and dS times a
// power of two f that brings a bound on it to 2^14 .. 2^15:
//   |P (dP - delta)| <= |dO_i| max_j |V_j| + |delta_i| =: b_i.
// dQ's f is its row's own; dK sums over queries, so its f is that of the
// largest b_i of the key/value head, which the dQ kernel leaves behind (a
// maximum, the same in any order).  |V_j| comes from window_v_norm_kernel.  The
// factors leave with the results' scale, at no cost in the loops.  What fp16
// still rounds away of a dS is 2^-25 / f, 2^-39 of the bound.
#pragma once

#include <cuda.h>

#include "window_args.cuh"
#include "window_fwd.cuh"
#include "window_ptx.cuh"

namespace vsa {

constexpr int kWbThreads = 384;
constexpr int kWbRows = 128;             // rows a CTA, and rows of a block it walks

template <int D>
struct WbSmem {
  static constexpr int kSlab = 128 * 128;
  static constexpr int kSlabs = D / 64;
  static constexpr int kBuf = kSlabs * kSlab;
  static constexpr int kOwn0 = 0, kOwn1 = kBuf;        // the CTA's own two tiles
  static constexpr int kASt = 3, kBSt = 2;             // stages of the walked tiles
  static constexpr int kA = 2 * kBuf, kB = kA + kASt * kBuf;
  static constexpr int kBar = kB + kBSt * kBuf;
  static constexpr int kNumBars = 24;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kXch = kMisc + 16;              // dq: float [2][128], delta and |dO|^2 between the warpgroups
  static constexpr int kStats = kXch;                  // dkv: (-lse * log2 e, -delta) of the walked queries,
                                                       // float [2 stages][2][128]
  static constexpr int kEnd = kStats + 2048;
  // what is left of a CTA's 227 KB, at most 1 KB, aligns the base
  static constexpr int kTotal = kEnd + 1024 < 232448 ? kEnd + 1024 : 232448;
  static_assert(kEnd + 256 <= 232448, "shared memory a CTA can have");
};

// The 1024-byte-aligned base of the buffers.  Dynamic shared memory begins on
// such a boundary; should it not, and the buffers not fit behind the next, the
// kernel reports it and does nothing.
template <int D>
__device__ __forceinline__ bool wb_base(const WinArgs& a, uint32_t raw, uint32_t& base) {
  uint32_t size;
  asm volatile("mov.u32 %0, %%dynamic_smem_size;" : "=r"(size));
  base = (raw + 1023u) & ~1023u;
  if (base - raw + WbSmem<D>::kEnd <= size) return true;
  if (threadIdx.x == 0) atomicCAS(a.err, 0u, 1u);
  return false;
}

// How the queries that see a key block are shared out: the first `heavy` key
// blocks (they hold first units, which every later query sees) among sh CTAs
// each, the others among sn <= sh.  A block with several CTAs gets its sums as float32
// partial tiles, [dK, dV][128 rows][D] a CTA, added in order by
// window_dkv_sum_kernel.
struct DkvSplit {
  int blocks, heavy, sh, sn;
  __host__ __device__ int ctas() const { return heavy * sh + (blocks - heavy) * sn; }
  // partial tiles of one (batch, key/value head): the first ones of its CTAs
  __host__ __device__ int tiles() const { return sn > 1 ? ctas() : sh > 1 ? heavy * sh : 0; }
};

// Stages this thread's row (D columns of TMEM at t) times f into the 128-row
// tile `buf`, swizzled as the TMA boxes are.
template <int D, bool F16>
__device__ __forceinline__ void stage_row(uint32_t t, uint32_t buf, int r, float f) {
#pragma unroll
  for (int q4 = 0; q4 < D / 32; ++q4) {
    uint32_t ov[32];
    tmem_ld32(t + 32u * q4, ov);
    tmem_wait_ld();
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e)
      pk[e] = pack_elem2<F16>(__uint_as_float(ov[2 * e]) * f, __uint_as_float(ov[2 * e + 1]) * f);
    const uint32_t at = buf + r * 128u + (q4 >> 1) * WbSmem<D>::kSlab;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      st_shared_v4(at + static_cast<uint32_t>(((q4 & 1) * 4 + e) ^ (r & 7)) * 16u, pk[4 * e], pk[4 * e + 1],
                   pk[4 * e + 2], pk[4 * e + 3]);
  }
}

// ------------------------------------------------------------------ range of fp16 operands
constexpr float kWbP = 4096.f;           // P's factor in the fp16 dK/dV kernel (log2: 12)

// The largest |V_j|^2 of a key/value head's chunk of keys that some query sees
// (the others may hold anything); sets the head's bound to 0 for the dQ kernel.
// Reads V once, D / 8 lanes a row, 4 rows in flight a lane (window_bwd_tokens: 3.3 us
// of latency; the whole gradient 139.6 us without the factors, 145.0 with).
template <int D>
__global__ void __launch_bounds__(256) window_v_norm_kernel(const __grid_constant__ WinArgs a) {
  constexpr int LPR = D / 8, R = 256 / LPR, U = 4;
  __shared__ float most[8];
  const int hk = blockIdx.y, b = blockIdx.z, len = win_len(a, b), start = win_start(a, b, len);
  const int j1 = static_cast<int>(1ll * a.Nk * (blockIdx.x + 1) / a.chunks);
  const uint16_t* v = a.v + b * a.vs[0] + hk * a.vs[2] + threadIdx.x % LPR * 8;
  // every CTA is resident from here on: the dQ kernel may set up beside them
  asm volatile("griddepcontrol.launch_dependents;");
  float m = 0.f;
  for (int j0 = static_cast<int>(1ll * a.Nk * blockIdx.x / a.chunks); j0 < j1; j0 += U * R) {
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * R + static_cast<int>(threadIdx.x) / LPR;
      x[u] = make_uint4(0u, 0u, 0u, 0u);
      if (j >= j1) continue;
      const KeyVis kv = key_vis(a, len, start, j);
      if (kv.lo < kv.hi) x[u] = __ldg(reinterpret_cast<const uint4*>(v + j * a.vs[1]));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = unpack_elem2<true>(w[e]);
        s = fmaf(f.x, f.x, fmaf(f.y, f.y, s));
      }
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      m = fmaxf(m, s);
    }
  }
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (threadIdx.x % 32 == 0) most[threadIdx.x / 32] = m;
  __syncthreads();
  if (threadIdx.x != 0) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, most[i]);
  const size_t head = static_cast<size_t>(b) * a.Hkv + hk;
  a.v_norms[head * a.chunks + blockIdx.x] = m;
  if (blockIdx.x == 0) a.grad_bound[head] = 0u;
}

// A lane's share of the largest |V_j|^2 of a key/value head.
__device__ __forceinline__ float lane_v_norm(const WinArgs& a, size_t head, int lane) {
  float m = 0.f;
  for (int c = lane; c < a.chunks; c += 32) m = fmaxf(m, a.v_norms[head * a.chunks + c]);
  return m;
}

// The power of two that brings a bound to [2^14, 2^15); 1 for 0, infinities and NaN.
__device__ __forceinline__ float grad_factor(unsigned int bound) {
  if (bound == 0u || bound >= 0x7f800000u) return 1.f;
  return __uint_as_float(static_cast<unsigned int>(min(268 - static_cast<int>(bound >> 23), 253)) << 23);
}

// ------------------------------------------------------------------ dQ
enum : int {
  DQ_OWN = 0, DQ_S = 1 /* [2] */, DQ_DP = 3, DQ_DP_FREE = 4, DQ_DS = 5 /* [2] */, DQ_S_FREE = 7 /* [2] */, DQ_OUT = 9,
  DQ_DRAIN = 10, DQ_K_FULL = 11, DQ_K_EMPTY = 14, DQ_V_FULL = 17, DQ_V_EMPTY = 19
};

// TMEM: two score buffers (dS of a warpgroup's 64 keys over the first 32
// columns of its half), dP, dQ.  Scores run two blocks ahead.  Warps: 0-3 and
// 4-7 elementwise (keys 0-63 and 64-127 of a block), 8 loads, 9 issues S, 10
// dP, 11 dQ.  About 2150 clk a block (window_bwd_wan5b: 680 us): 64 KB of K and V
// have to enter shared memory for 1536 clk of MMA that read it too.  The
// warpgroups on alternate blocks instead: 725 us.
template <int D, bool F16>
__global__ void __launch_bounds__(kWbThreads, 1)
    window_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmG,
                     const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmDQ, const __grid_constant__ WinArgs a) {
  using L = WbSmem<D>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint32_t base;
  if (!wb_base<D>(a, raw, base)) return;
  unsigned char* sp = smem_raw + (base - raw);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sp + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sp + L::kMisc + 4);
  auto bar = [&](int id) -> uint32_t { return base + L::kBar + 8u * static_cast<uint32_t>(id); };

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int h = blockIdx.y, b = blockIdx.z, hk = h / a.group;
  const int i0 = (gridDim.x - 1 - blockIdx.x) * kWbRows;
  const int len = win_len(a, b), start = win_start(a, b, len);
  const WinBlocks wb = win_blocks(a, len, start, i0, min(i0 + kWbRows, a.Nq) - 1);
  const int n = wb.count();

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kNumBars; ++i) {
      uint32_t cnt = 1;
      if (i == DQ_DP_FREE || i == DQ_DS || i == DQ_DS + 1) cnt = 256;
      if (i == DQ_DRAIN) cnt = 3;
      mbar_init(bar(i), cnt);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 11) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tDP = tmem + 256, tDQ = tmem + 384;

  if (warp == 8) {
    // ====================================================== TMA producer
    if (lane == 0 && n > 0) {
      mbar_arrive_expect_tx(bar(DQ_OWN), 2 * L::kBuf);
      for (int sl = 0; sl < L::kSlabs; ++sl) {
        tma_load_4d(base + L::kOwn0 + sl * L::kSlab, &tmQ, bar(DQ_OWN), sl * 64, i0, h, b);
        tma_load_4d(base + L::kOwn1 + sl * L::kSlab, &tmG, bar(DQ_OWN), sl * 64, i0, h, b);
      }
      int kd = 0, vd = 0;                              // loads issued
      for (int j = 0; j < n; ++j) {
        const int c0 = wb.block(j) * kWfKeys;
        const int ks = j % L::kASt, vs = j % L::kBSt;
        if (j >= L::kASt && !mbar_wait(bar(DQ_K_EMPTY + ks), (j / L::kASt - 1) & 1, abort_flag, a.err)) break;
        kd = j + 1;
        mbar_arrive_expect_tx(bar(DQ_K_FULL + ks), L::kBuf);
        for (int sl = 0; sl < L::kSlabs; ++sl)
          tma_load_4d(base + L::kA + ks * L::kBuf + sl * L::kSlab, &tmK, bar(DQ_K_FULL + ks), sl * 64, c0, hk, b);
        if (j >= L::kBSt && !mbar_wait(bar(DQ_V_EMPTY + vs), (j / L::kBSt - 1) & 1, abort_flag, a.err)) break;
        vd = j + 1;
        mbar_arrive_expect_tx(bar(DQ_V_FULL + vs), L::kBuf);
        for (int sl = 0; sl < L::kSlabs; ++sl)
          tma_load_4d(base + L::kB + vs * L::kBuf + sl * L::kSlab, &tmV, bar(DQ_V_FULL + vs), sl * 64, c0, hk, b);
      }
      // let every issued copy land before the CTA can exit
      for (int j = max(0, kd - L::kASt); j < kd; ++j)
        mbar_wait(bar(DQ_K_FULL + j % L::kASt), (j / L::kASt) & 1, nullptr, a.err);
      for (int j = max(0, vd - L::kBSt); j < vd; ++j)
        mbar_wait(bar(DQ_V_FULL + j % L::kBSt), (j / L::kBSt) & 1, nullptr, a.err);
      mbar_wait(bar(DQ_OWN), 0, nullptr, a.err);
    }
    __syncwarp();
  } else if (warp >= 9) {
    // ====================================================== MMA issuers
    constexpr uint32_t idS = idesc_f16kind_f32(128, 128, false, F16);
    constexpr uint32_t idQ = idesc_f16kind_f32(128, D, true, F16);
    bool ok = n == 0 || __all_sync(0xffffffffu, mbar_wait(bar(DQ_OWN), 0, abort_flag, a.err));
    for (int j = 0; j < n && ok; ++j) {
      const int ks = j % L::kASt, vs = j % L::kBSt, sb = j & 1;
      const uint32_t kb = base + L::kA + ks * L::kBuf, vb = base + L::kB + vs * L::kBuf;
      if (warp == 9) {                                 // S(j) once K(j) is in and dQ(j-2) has read dS(j-2)
        ok = __all_sync(0xffffffffu, mbar_wait(bar(DQ_K_FULL + ks), (j / L::kASt) & 1, abort_flag, a.err) &&
                                         (j < 2 || mbar_wait(bar(DQ_S_FREE + sb), ((j >> 1) - 1) & 1, abort_flag, a.err)));
      } else if (warp == 10) {                         // dP(j) once V(j) is in and dP(j-1) has been read
        ok = __all_sync(0xffffffffu, mbar_wait(bar(DQ_V_FULL + vs), (j / L::kBSt) & 1, abort_flag, a.err) &&
                                         (j < 1 || mbar_wait(bar(DQ_DP_FREE), (j - 1) & 1, abort_flag, a.err)));
      } else {                                         // dQ += dS(j) K(j)
        ok = __all_sync(0xffffffffu, mbar_wait(bar(DQ_K_FULL + ks), (j / L::kASt) & 1, abort_flag, a.err) &&
                                         mbar_wait(bar(DQ_DS + sb), (j >> 1) & 1, abort_flag, a.err));
      }
      if (!ok) break;
      tc_fence_after();
      if (elect_one_sync()) {
        if (warp == 9) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const int off = (kk / 4) * L::kSlab + (kk % 4) * 32;
            mma_ss(tmem + 128u * sb, smem_desc_sw128(base + L::kOwn0 + off, 16, 1024), smem_desc_sw128(kb + off, 16, 1024),
                   idS, kk > 0 ? 1u : 0u);
          }
          mma_commit(bar(DQ_S + sb));
        } else if (warp == 10) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const int off = (kk / 4) * L::kSlab + (kk % 4) * 32;
            mma_ss(tDP, smem_desc_sw128(base + L::kOwn1 + off, 16, 1024), smem_desc_sw128(vb + off, 16, 1024), idS,
                   kk > 0 ? 1u : 0u);
          }
          mma_commit(bar(DQ_DP));
          mma_commit(bar(DQ_V_EMPTY + vs));
        } else {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)               // 16 keys a step: 8 columns of a warpgroup's 32
            mma_ts(tDQ, tmem + 128u * sb + 64u * (kk / 4) + 8u * (kk % 4), smem_desc_sw128(kb + kk * 2048, L::kSlab, 1024),
                   idQ, (j > 0 || kk > 0) ? 1u : 0u);
          mma_commit(bar(DQ_K_EMPTY + ks));
          mma_commit(bar(DQ_S_FREE + sb));
          if (j == n - 1) mma_commit(bar(DQ_OUT));
        }
      }
      __syncwarp();
    }
    if (elect_one_sync()) mma_commit(bar(DQ_DRAIN));
    __syncwarp();
    mbar_wait(bar(DQ_DRAIN), 0, nullptr, a.err);
  } else {
    // ====================================================== elementwise
    const int w = warp / 4, r = threadIdx.x % 128;
    const int i = i0 + r;
    const uint32_t lane_base = static_cast<uint32_t>((warp % 4) * 32) << 16;
    RowVis vis{0, 0, 0};
    float lse2 = 0.f, delta = 0.f, g2 = 0.f;           // g2: |dO_i|^2 (fp16)
    const size_t row = (static_cast<size_t>(b) * a.Hq + h) * a.Nq + i, head = static_cast<size_t>(b) * a.Hkv + hk;
    if (i < a.Nq) {
      vis = row_vis(a, len, start + i);
      const float ls = a.lse[row];
      lse2 = ls == -INFINITY ? 0.f : ls * 1.4426950408889634f;
      // delta: this warpgroup's half of the channels, then both halves
      const uint4* op = reinterpret_cast<const uint4*>(a.o + b * a.os[0] + i * a.os[1] + h * a.os[2]) + w * (D / 16);
      const uint4* gp = reinterpret_cast<const uint4*>(a.d_o + b * a.dos[0] + i * a.dos[1] + h * a.dos[2]) + w * (D / 16);
#pragma unroll
      for (int e = 0; e < D / 16; ++e) {
        const uint4 x = __ldg(op + e), g = __ldg(gp + e);
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, gs[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float2 xf = unpack_elem2<F16>(xs[u]), gf = unpack_elem2<F16>(gs[u]);
          delta = fmaf(xf.x, gf.x, fmaf(xf.y, gf.y, delta));
          if (F16) g2 = fmaf(gf.x, gf.x, fmaf(gf.y, gf.y, g2));
        }
      }
    }
    float* xch = reinterpret_cast<float*>(sp + L::kXch);
    if (w == 1) {
      xch[r] = delta;
      if (F16) xch[128 + r] = g2;
    }
    named_bar_sync(1, 256);
    if (w == 0) {
      delta += xch[r];
      xch[r] = delta;
      if (F16) xch[128 + r] = g2 += xch[128 + r];
    }
    named_bar_sync(1, 256);
    delta = xch[r];
    if (w == 0 && i < a.Nq) a.delta[row] = delta;
    float f = 1.f;                                     // dS's factor
    if (F16) {
      asm volatile("griddepcontrol.wait;" ::: "memory");           // for window_v_norm_kernel's results
      float v2 = lane_v_norm(a, head, lane);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) v2 = fmaxf(v2, __shfl_xor_sync(0xffffffffu, v2, o));
      const unsigned int bound = __float_as_uint(sqrtf(xch[128 + r] * v2) + fabsf(delta));
      f = grad_factor(bound);
      if (w == 0) {
        const bool sees = vis.hi > vis.lo || vis.first > 0;        // (a query that sees nothing may hold anything)
        const unsigned int most = __reduce_max_sync(0xffffffffu, sees ? bound : 0u);
        if (lane == 0) atomicMax(a.grad_bound + head, most);
      }
    }

    bool ok = true;
    const uint64_t sc2 = f2_pack(a.scale_log2, a.scale_log2), nl2 = f2_pack(-lse2, -lse2), f2 = f2_pack(f, f),
                   nd2 = f2_pack(-delta * f, -delta * f);
    for (int j = 0; j < n; ++j) {
      const int c0 = wb.block(j) * kWfKeys, sb = j & 1;
      const uint32_t tS = tmem + lane_base + 128u * sb + 64u * w, tP = tDP + lane_base + 64u * w;
      const bool row_full = i >= a.Nq || c0 + kWfKeys <= vis.first || (c0 >= vis.lo && c0 + kWfKeys <= vis.hi);
      const bool masked = __any_sync(0xffffffffu, !row_full);
      // Keys that no row of the CTA sees may hold anything: zero their K rows
      // (0 * NaN would reach dQ).
      if ((c0 + kWfKeys > wb.hi || c0 < wb.lo) && c0 + kWfKeys > wb.first) {
        const int ks = j % L::kASt;
        if (!__all_sync(0xffffffffu, mbar_wait(bar(DQ_K_FULL + ks), (j / L::kASt) & 1, abort_flag, a.err))) {
          ok = false;
          break;
        }
        if (w == 0) zero_unseen<D>(base + L::kA + ks * L::kBuf, c0, wb.first, wb.lo, wb.hi, r);
        fence_proxy_async_smem();
      }
      if (!__all_sync(0xffffffffu, mbar_wait(bar(DQ_S + sb), (j >> 1) & 1, abort_flag, a.err))) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t x[64], g[64];
      tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
      tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&x[32]));
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        float z0, z1;
        f2_unpack(f2_fma(f2_pack(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), sc2, nl2), z0, z1);
        x[2 * e] = __float_as_uint(ex2_approx(z0));
        x[2 * e + 1] = __float_as_uint(ex2_approx(z1));
      }
      if (!__all_sync(0xffffffffu, mbar_wait(bar(DQ_DP), j & 1, abort_flag, a.err))) {
        ok = false;
        break;
      }
      tc_fence_after();
      tmem_ld32(tP, *reinterpret_cast<uint32_t(*)[32]>(&g[0]));
      tmem_ld32(tP + 32, *reinterpret_cast<uint32_t(*)[32]>(&g[32]));
      tmem_wait_ld();
      tc_fence_before();
      mbar_arrive(bar(DQ_DP_FREE));
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        float d0, d1;
        const uint64_t dp = f2_pack(__uint_as_float(g[2 * e]), __uint_as_float(g[2 * e + 1]));
        f2_unpack(F16 ? f2_fma(dp, f2, nd2) : f2_add(dp, nd2), d0, d1);
        x[2 * e] = __float_as_uint(__uint_as_float(x[2 * e]) * d0);
        x[2 * e + 1] = __float_as_uint(__uint_as_float(x[2 * e + 1]) * d1);
      }
      if (masked) {
        uint32_t mw[4];
        vis_words(vis, c0, mw);
        const uint32_t m0 = w == 0 ? mw[0] : mw[2], m1 = w == 0 ? mw[1] : mw[3];
#pragma unroll
        for (int e = 0; e < 64; ++e)
          if (!(((e < 32 ? m0 : m1) >> (e & 31)) & 1u)) x[e] = 0u;
      }
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] = pack_elem2<F16>(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
      tmem_st32(tS, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar(DQ_DS + sb));
    }
    // ---- epilogue: warpgroup 0 writes dQ through Q's buffer
    if (ok && n > 0) ok = __all_sync(0xffffffffu, mbar_wait(bar(DQ_OUT), 0, abort_flag, a.err));
    tc_fence_after();
    if (w == 0) {
      if (n > 0) {
        if (ok) stage_row<D, F16>(tDQ + lane_base, base + L::kOwn0, r, a.scale / f);
        fence_proxy_async_smem();
        named_bar_sync(2, 128);
        if (ok && r == 0) {
          for (int sl = 0; sl < L::kSlabs; ++sl)
            tma_store_4d(&tmDQ, base + L::kOwn0 + sl * L::kSlab, sl * 64, i0, h, b);
          bulk_commit_group();
          bulk_wait_group_read0();
        }
      } else if (i < a.Nq) {
        uint4* o = reinterpret_cast<uint4*>(a.dq + b * a.dqs[0] + i * a.dqs[1] + h * a.dqs[2]);
#pragma unroll
        for (int e = 0; e < D / 8; ++e) o[e] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 11) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ dK, dV
enum : int {
  DK_OWN = 0, DK_S = 1, DK_P = 2 /* [half] */, DK_DP = 4, DK_DS = 5, DK_OUT = 6 /* [2] */, DK_DRAIN = 8,
  DK_Q_FULL = 9 /* [3] */, DK_Q_EMPTY = 12, DK_G_FULL = 15 /* [2] */, DK_G_EMPTY = 17, DK_ST_FULL = 19, DK_ST_EMPTY = 21
};

// The CTA's 128 keys are the rows, the queries of a block the columns.  TMEM:
// S^T, dP^T, dV, dK; P^T and dS^T of a warpgroup's 64 queries over the first
// 32 columns of its half.  One warp issues dV(j) and right behind it S(j+1),
// another dK(j) and dP(j+1): the next scores are made while the elementwise
// warps finish dS.  P^T is released in two parts, so dV starts before the
// exponentials end.  Warps: 0-7 elementwise, 8 loads, 9 fetches LSE and delta
// of the walked queries, 10 issues S and dV, 11 dP and dK.
template <int D, bool F16, bool SHARED>
__global__ void __launch_bounds__(kWbThreads, 1)
    window_dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmG,
                      const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ CUtensorMap tmDK, const __grid_constant__ CUtensorMap tmDV,
                      const __grid_constant__ WinArgs a, const DkvSplit ds, float* part) {
  using L = WbSmem<D>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint32_t base;
  if (!wb_base<D>(a, raw, base)) return;
  unsigned char* sp = smem_raw + (base - raw);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sp + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sp + L::kMisc + 4);
  float* stats = reinterpret_cast<float*>(sp + L::kStats);
  auto bar = [&](int id) -> uint32_t { return base + L::kBar + 8u * static_cast<uint32_t>(id); };

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int hk = blockIdx.y, b = blockIdx.z;
  // first keys first: they may be seen by every query
  int blk = blockIdx.x, S = 1, sp_i = 0;               // S: CTAs of this key block (SHARED: some have several)
  if (SHARED) {
    const int x = blockIdx.x - ds.heavy * ds.sh;
    const bool hv = x < 0;
    S = hv ? ds.sh : ds.sn;
    blk = hv ? blockIdx.x / S : ds.heavy + x / S;
    sp_i = hv ? blockIdx.x % S : x % S;
  }
  const int c0 = blk * kWbRows;
  const int len = win_len(a, b), start = win_start(a, b, len);
  const float fds = F16 ? grad_factor(a.grad_bound[static_cast<size_t>(b) * a.Hkv + hk]) : 1.f;      // dS's factor
  // queries that see some key of [c0, c1): one range of rows, [qlo, qhi)
  int qb0 = 0, nq = 0;
  if (c0 < len) {
    const int c1 = min(c0 + kWbRows, len);
    const long long p0 = static_cast<long long>(c0 / a.unit) * a.unit;
    const long long p1 = c0 < a.sink_tok ? (1ll << 40) : ((c1 - 1) / a.unit + static_cast<long long>(a.window)) * a.unit;
    const long long qlo = max(p0 - start, 0ll), qhi = min(p1 - start, static_cast<long long>(a.Nq));
    if (qhi > qlo) {
      qb0 = static_cast<int>(qlo / kWbRows);
      nq = static_cast<int>((qhi + kWbRows - 1) / kWbRows) - qb0;
    }
  }
  const int n_all = nq * a.group;
  const int j0 = SHARED ? static_cast<int>(static_cast<long long>(n_all) * sp_i / S) : 0;
  const int n = SHARED ? static_cast<int>(static_cast<long long>(n_all) * (sp_i + 1) / S) - j0 : n_all;   // this CTA's walk

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kNumBars; ++i) {
      uint32_t cnt = 1;
      if (i == DK_P || i == DK_P + 1 || i == DK_DS || i == DK_ST_EMPTY || i == DK_ST_EMPTY + 1) cnt = 256;
      if (i == DK_DRAIN || (i >= DK_Q_EMPTY && i < DK_Q_EMPTY + 3) || (i >= DK_G_EMPTY && i < DK_G_EMPTY + 2)) cnt = 2;
      if (i == DK_ST_FULL || i == DK_ST_FULL + 1) cnt = 32;
      mbar_init(bar(i), cnt);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 11) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tS = tmem, tDP = tmem + 128, tDV = tmem + 256, tDK = tmem + 384;
  // walked block j: query head hk * group + (j0 + j) / nq, rows from (qb0 + (j0 + j) % nq) * 128
  const int h_first = hk * a.group + (SHARED && nq > 0 ? j0 / nq : 0), q_first = SHARED && nq > 0 ? j0 % nq : 0;

  if (warp == 8) {
    // ====================================================== TMA producer
    if (lane == 0 && n > 0) {
      mbar_arrive_expect_tx(bar(DK_OWN), 2 * L::kBuf);
      for (int sl = 0; sl < L::kSlabs; ++sl) {
        tma_load_4d(base + L::kOwn0 + sl * L::kSlab, &tmK, bar(DK_OWN), sl * 64, c0, hk, b);
        tma_load_4d(base + L::kOwn1 + sl * L::kSlab, &tmV, bar(DK_OWN), sl * 64, c0, hk, b);
      }
      int qd = 0, gd = 0, h = h_first, qi = q_first;
      for (int j = 0; j < n; ++j) {
        const int st = j & 1, qs = j % L::kASt, i0 = (qb0 + qi) * kWbRows;
        if (j >= L::kASt && !mbar_wait(bar(DK_Q_EMPTY + qs), (j / L::kASt - 1) & 1, abort_flag, a.err)) break;
        qd = j + 1;
        mbar_arrive_expect_tx(bar(DK_Q_FULL + qs), L::kBuf);
        for (int sl = 0; sl < L::kSlabs; ++sl)
          tma_load_4d(base + L::kA + qs * L::kBuf + sl * L::kSlab, &tmQ, bar(DK_Q_FULL + qs), sl * 64, i0, h, b);
        if (j >= 2 && !mbar_wait(bar(DK_G_EMPTY + st), ((j >> 1) - 1) & 1, abort_flag, a.err)) break;
        gd = j + 1;
        mbar_arrive_expect_tx(bar(DK_G_FULL + st), L::kBuf);
        for (int sl = 0; sl < L::kSlabs; ++sl)
          tma_load_4d(base + L::kB + st * L::kBuf + sl * L::kSlab, &tmG, bar(DK_G_FULL + st), sl * 64, i0, h, b);
        if (++qi == nq) { qi = 0; ++h; }
      }
      for (int j = max(0, qd - L::kASt); j < qd; ++j)
        mbar_wait(bar(DK_Q_FULL + j % L::kASt), (j / L::kASt) & 1, nullptr, a.err);
      for (int j = max(0, gd - 2); j < gd; ++j) mbar_wait(bar(DK_G_FULL + (j & 1)), (j >> 1) & 1, nullptr, a.err);
      mbar_wait(bar(DK_OWN), 0, nullptr, a.err);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ====================================================== LSE and delta
    int h = h_first, qi = q_first;
    for (int j = 0; j < n; ++j) {
      const int st = j & 1, i0 = (qb0 + qi) * kWbRows;
      const size_t row0 = (static_cast<size_t>(b) * a.Hq + h) * a.Nq;
      float ls[4], de[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = i0 + 32 * e + lane;
        ls[e] = i < a.Nq ? a.lse[row0 + i] : 0.f;
        de[e] = i < a.Nq ? a.delta[row0 + i] : 0.f;
      }
      if (j >= 2 &&
          !__all_sync(0xffffffffu, mbar_wait(bar(DK_ST_EMPTY + st), ((j >> 1) - 1) & 1, abort_flag, a.err)))
        break;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        stats[st * 256 + 32 * e + lane] = (ls[e] == -INFINITY ? 0.f : -ls[e] * 1.4426950408889634f) + (F16 ? 12.f : 0.f);
        stats[st * 256 + 128 + 32 * e + lane] = F16 ? -de[e] * (fds / kWbP) : -de[e];
      }
      mbar_arrive(bar(DK_ST_FULL + st));
      if (++qi == nq) { qi = 0; ++h; }
    }
  } else if (warp >= 10) {
    // ====================================================== MMA issuers
    constexpr uint32_t idS = idesc_f16kind_f32(128, 128, false, F16);
    constexpr uint32_t idO = idesc_f16kind_f32(128, D, true, F16);
    const bool first = warp == 10;                     // S, dV; else dP, dK
    bool ok = n == 0 || __all_sync(0xffffffffu, mbar_wait(bar(DK_OWN), 0, abort_flag, a.err));
    auto wait_in = [&](int j, bool g) {                // Q(j) or dO(j) has landed
      ok = __all_sync(0xffffffffu, g ? mbar_wait(bar(DK_G_FULL + (j & 1)), (j >> 1) & 1, abort_flag, a.err)
                                     : mbar_wait(bar(DK_Q_FULL + j % L::kASt), (j / L::kASt) & 1, abort_flag, a.err));
    };
    // (elected lane) S(j) = K Q(j)^T, or dP(j) = V dO(j)^T
    auto make = [&](int j) {
      const uint32_t own = base + (first ? L::kOwn0 : L::kOwn1);
      const uint32_t in = base + (first ? L::kA + (j % L::kASt) * L::kBuf : L::kB + (j & 1) * L::kBuf);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const int off = (kk / 4) * L::kSlab + (kk % 4) * 32;
        mma_ss(first ? tS : tDP, smem_desc_sw128(own + off, 16, 1024), smem_desc_sw128(in + off, 16, 1024), idS,
               kk > 0 ? 1u : 0u);
      }
      mma_commit(bar(first ? DK_S : DK_DP));
      mma_commit(bar(first ? DK_Q_EMPTY + j % L::kASt : DK_G_EMPTY + (j & 1)));
    };
    if (ok && n > 0) {
      wait_in(0, !first);
      if (ok) {
        tc_fence_after();
        if (elect_one_sync()) make(0);
        __syncwarp();
      }
    }
    for (int j = 0; j < n && ok; ++j) {
      // The next block's scores are queued right behind this block's product:
      // their operand is waited for before it, since a barrier test behind
      // queued MMAs waits for them to drain -- and then the other warp's MMAs
      // would come between (dK and dP before S: 3300 clk a block).
      const int st = j & 1;
      wait_in(j, first);
      if (first) {
        const uint32_t gb = base + L::kB + st * L::kBuf;
#pragma unroll
        for (int hf = 0; hf < 2 && ok; ++hf) {
          if (hf == 1 && j + 1 < n) wait_in(j + 1, false);
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(DK_P + hf), j & 1, abort_flag, a.err));
          if (!ok) break;
          tc_fence_after();
          if (elect_one_sync()) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int kk = 4 * (e >> 1) + 2 * hf + (e & 1);      // queries 16 kk .. 16 kk + 15
              mma_ts(tDV, tS + 64u * (kk / 4) + 8u * (kk % 4), smem_desc_sw128(gb + kk * 2048, L::kSlab, 1024), idO,
                     (j > 0 || hf > 0 || e > 0) ? 1u : 0u);
            }
            if (hf == 1) {
              if (j + 1 < n) make(j + 1);
              mma_commit(bar(DK_G_EMPTY + st));
              if (j == n - 1) mma_commit(bar(DK_OUT));
            }
          }
          __syncwarp();
        }
      } else {
        if (ok && j + 1 < n) wait_in(j + 1, true);
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(DK_DS), j & 1, abort_flag, a.err));
        if (!ok) break;
        tc_fence_after();
        if (elect_one_sync()) {
          const uint32_t qb = base + L::kA + (j % L::kASt) * L::kBuf;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts(tDK, tDP + 64u * (kk / 4) + 8u * (kk % 4), smem_desc_sw128(qb + kk * 2048, L::kSlab, 1024), idO,
                   (j > 0 || kk > 0) ? 1u : 0u);
          if (j + 1 < n) make(j + 1);
          mma_commit(bar(DK_Q_EMPTY + j % L::kASt));
          if (j == n - 1) mma_commit(bar(DK_OUT + 1));
        }
        __syncwarp();
      }
    }
    if (elect_one_sync()) mma_commit(bar(DK_DRAIN));
    __syncwarp();
    mbar_wait(bar(DK_DRAIN), 0, nullptr, a.err);
  } else {
    // ====================================================== elementwise
    const int w = warp / 4, r = threadIdx.x % 128;
    const int key = c0 + r;
    const uint32_t lane_base = static_cast<uint32_t>((warp % 4) * 32) << 16;
    const uint32_t tSw = tS + lane_base + 64u * w, tPw = tDP + lane_base + 64u * w;
    // the query rows that see this key: [qlo, qhi)
    const KeyVis rows = key_vis(a, len, start, key);
    const int qlo = rows.lo, qhi = rows.hi;
    bool ok = true;
    const uint64_t sc2 = f2_pack(a.scale_log2, a.scale_log2), fd2 = f2_pack(fds / kWbP, fds / kWbP);
    const float fo = w == 0 ? (F16 ? 1.f / kWbP : 1.f) : a.scale / fds;        // of dV, of dK
    int qi = q_first;
    for (int j = 0; j < n; ++j) {
      const int st = j & 1, i0 = (qb0 + qi) * kWbRows;
      if (++qi == nq) qi = 0;
      const bool masked = __any_sync(0xffffffffu, qlo > i0 || qhi < i0 + kWbRows);
      // Queries that see nothing may hold anything: zero their Q and dO rows.
      // They are the rows before position 0, and those whose window lies
      // behind the last key.
      const int il = min(i0 + kWbRows, a.Nq) - 1;
      if (start + i0 < 0 || (masked && row_vis(a, len, start + il).hi == row_vis(a, len, start + il).lo &&
                             row_vis(a, len, start + il).first == 0)) {
        if (!__all_sync(0xffffffffu, mbar_wait(bar(DK_Q_FULL + j % L::kASt), (j / L::kASt) & 1, abort_flag, a.err) &&
                                         mbar_wait(bar(DK_G_FULL + st), (j >> 1) & 1, abort_flag, a.err))) {
          ok = false;
          break;
        }
        // the live rows are those from position 0 on whose window begins before the end
        // of the keys (with first units, all of them); one range of the block
        const int at0 = max(0, -(start + i0));
        int n_live = 0;
        for (int e = lane; e < kWbRows; e += 32) {
          const RowVis v = row_vis(a, len, start + i0 + e);
          n_live += __popc(__ballot_sync(0xffffffffu, v.hi > v.lo || v.first > 0));
        }
        zero_unseen<D>(base + (w == 0 ? L::kA + (j % L::kASt) * L::kBuf : L::kB + st * L::kBuf), 0, 0, at0, at0 + n_live, r);
        fence_proxy_async_smem();
      }
      if (!__all_sync(0xffffffffu, mbar_wait(bar(DK_ST_FULL + st), (j >> 1) & 1, abort_flag, a.err) &&
                                       mbar_wait(bar(DK_S), j & 1, abort_flag, a.err))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const float4* nl = reinterpret_cast<const float4*>(stats + st * 256 + 64 * w);
      const float4* nd = reinterpret_cast<const float4*>(stats + st * 256 + 128 + 64 * w);
      uint32_t x[64];
      tmem_ld32(tSw, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
      tmem_ld32(tSw + 32, *reinterpret_cast<uint32_t(*)[32]>(&x[32]));
      tmem_wait_ld();
      uint32_t m0 = ~0u, m1 = ~0u;
      if (masked) {
        const int q0 = i0 + 64 * w;
        m0 = low_bits(qhi - q0) & ~low_bits(qlo - q0);
        m1 = low_bits(qhi - q0 - 32) & ~low_bits(qlo - q0 - 32);
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 8 * hf; e < 8 * hf + 8; ++e) {
          const float4 l4 = nl[e];
          float z0, z1, z2, z3;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(x[4 * e]), __uint_as_float(x[4 * e + 1])), sc2, f2_pack(l4.x, l4.y)), z0, z1);
          f2_unpack(f2_fma(f2_pack(__uint_as_float(x[4 * e + 2]), __uint_as_float(x[4 * e + 3])), sc2, f2_pack(l4.z, l4.w)), z2, z3);
          x[4 * e] = __float_as_uint(ex2_approx(z0));
          x[4 * e + 1] = __float_as_uint(ex2_approx(z1));
          x[4 * e + 2] = __float_as_uint(ex2_approx(z2));
          x[4 * e + 3] = __float_as_uint(ex2_approx(z3));
        }
        if (masked) {
#pragma unroll
          for (int e = 32 * hf; e < 32 * hf + 32; ++e)
            if (!(((hf == 0 ? m0 : m1) >> (e & 31)) & 1u)) x[e] = 0u;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e)
          pk[e] = pack_elem2<F16>(__uint_as_float(x[32 * hf + 2 * e]), __uint_as_float(x[32 * hf + 2 * e + 1]));
        tmem_st16(tSw + 16u * hf, pk);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(DK_P + hf));
      }
      if (!__all_sync(0xffffffffu, mbar_wait(bar(DK_DP), j & 1, abort_flag, a.err))) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t g[64], pk[32];
      tmem_ld32(tPw, *reinterpret_cast<uint32_t(*)[32]>(&g[0]));
      tmem_ld32(tPw + 32, *reinterpret_cast<uint32_t(*)[32]>(&g[32]));
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float4 d4 = nd[e];
        float d0, d1, d2, d3;
        const uint64_t dpa = f2_pack(__uint_as_float(g[4 * e]), __uint_as_float(g[4 * e + 1]));
        const uint64_t dpb = f2_pack(__uint_as_float(g[4 * e + 2]), __uint_as_float(g[4 * e + 3]));
        f2_unpack(F16 ? f2_fma(dpa, fd2, f2_pack(d4.x, d4.y)) : f2_add(dpa, f2_pack(d4.x, d4.y)), d0, d1);
        f2_unpack(F16 ? f2_fma(dpb, fd2, f2_pack(d4.z, d4.w)) : f2_add(dpb, f2_pack(d4.z, d4.w)), d2, d3);
        if (masked) {                                  // (P is 0 there, but dP may not be finite)
          const uint32_t mm = (e < 8 ? m0 : m1) >> ((4 * e) & 31);
          if (!(mm & 1u)) d0 = 0.f;
          if (!(mm & 2u)) d1 = 0.f;
          if (!(mm & 4u)) d2 = 0.f;
          if (!(mm & 8u)) d3 = 0.f;
        }
        pk[2 * e] = pack_elem2<F16>(__uint_as_float(x[4 * e]) * d0, __uint_as_float(x[4 * e + 1]) * d1);
        pk[2 * e + 1] = pack_elem2<F16>(__uint_as_float(x[4 * e + 2]) * d2, __uint_as_float(x[4 * e + 3]) * d3);
      }
      tmem_st32(tPw, pk);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar(DK_DS));
      mbar_arrive(bar(DK_ST_EMPTY + st));
    }
    // ---- epilogue: warpgroup 0 writes dV through V's buffer, 1 dK through K's
    if (SHARED && S > 1) {
      if (n > 0 && ok)
        ok = __all_sync(0xffffffffu, mbar_wait(bar(DK_OUT), 0, abort_flag, a.err) &&
                                         mbar_wait(bar(DK_OUT + 1), 0, abort_flag, a.err));
      tc_fence_after();
      float* op = part + ((static_cast<size_t>(b) * a.Hkv + hk) * ds.tiles() + blockIdx.x) * (2 * 128 * D) +
                  (w == 0 ? 128 * D : 0) + r * D;
#pragma unroll
      for (int q4 = 0; q4 < D / 32; ++q4) {
        uint32_t ov[32];
        if (n > 0) {
          tmem_ld32((w == 0 ? tDV : tDK) + lane_base + 32u * q4, ov);
          tmem_wait_ld();
        }
        if (ok) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            reinterpret_cast<uint4*>(op + 32 * q4)[e] =
                n > 0 ? make_uint4(ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]) : make_uint4(0u, 0u, 0u, 0u);
        }
      }
    } else if (n > 0) {
      if (ok)
        ok = __all_sync(0xffffffffu, mbar_wait(bar(DK_OUT), 0, abort_flag, a.err) &&
                                         mbar_wait(bar(DK_OUT + 1), 0, abort_flag, a.err));
      tc_fence_after();
      const uint32_t buf = base + (w == 0 ? L::kOwn1 : L::kOwn0);
      if (ok) stage_row<D, F16>((w == 0 ? tDV : tDK) + lane_base, buf, r, fo);
      fence_proxy_async_smem();
      named_bar_sync(1 + w, 128);
      if (ok && r == 0) {
        for (int sl = 0; sl < L::kSlabs; ++sl)
          tma_store_4d(w == 0 ? &tmDV : &tmDK, buf + sl * L::kSlab, sl * 64, c0, hk, b);
        bulk_commit_group();
        bulk_wait_group_read0();
      }
    } else if (key < a.Nk) {                           // keys that no query sees
      uint4* o = reinterpret_cast<uint4*>(w == 0 ? a.dv + b * a.dvs[0] + key * a.dvs[1] + hk * a.dvs[2]
                                                 : a.dk + b * a.dks[0] + key * a.dks[1] + hk * a.dks[2]);
#pragma unroll
      for (int e = 0; e < D / 8; ++e) o[e] = make_uint4(0u, 0u, 0u, 0u);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 11) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// dK and dV rows of the key blocks that several CTAs shared: their partial
// tiles added in order.  One thread 4 channels of a row.
template <int D, bool F16>
__global__ void __launch_bounds__(256) window_dkv_sum_kernel(const __grid_constant__ WinArgs a, const DkvSplit ds,
                                                             const float* part) {
  const int blk = blockIdx.x / (D / 4), hk = blockIdx.y, b = blockIdx.z;     // D / 4 CTAs of 256 a block: 2 x 128 x D / 4
  const bool hv = blk < ds.heavy;
  const int S = hv ? ds.sh : ds.sn;
  const int tile = hv ? blk * S : ds.heavy * ds.sh + (blk - ds.heavy) * S;
  const int at = (blockIdx.x % (D / 4)) * 256 + threadIdx.x;                         // float4 of a tile
  const float4* p = reinterpret_cast<const float4*>(
                        part + ((static_cast<size_t>(b) * a.Hkv + hk) * ds.tiles() + tile) * (2 * 128 * D)) + at;
  float4 s = p[0];
  for (int i = 1; i < S; ++i) {
    const float4 v = p[static_cast<size_t>(i) * (2 * 128 * D / 4)];
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
  const bool is_v = at >= 128 * D / 4;
  const int e = is_v ? at - 128 * D / 4 : at;
  const int key = blk * kWbRows + e / (D / 4), ch = (e % (D / 4)) * 4;
  if (key >= a.Nk) return;
  const float f = !F16 ? (is_v ? 1.f : a.scale)
                       : is_v ? 1.f / kWbP : a.scale / grad_factor(a.grad_bound[static_cast<size_t>(b) * a.Hkv + hk]);
  uint16_t* o = is_v ? a.dv + b * a.dvs[0] + key * a.dvs[1] + hk * a.dvs[2] : a.dk + b * a.dks[0] + key * a.dks[1] + hk * a.dks[2];
  *reinterpret_cast<uint2*>(o + ch) = make_uint2(pack_elem2<F16>(s.x * f, s.y * f), pack_elem2<F16>(s.z * f, s.w * f));
}

}  // namespace vsa

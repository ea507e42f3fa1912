// window_fwd.cuh -- window attention forward for sm_100a.
//
// One CTA = 256 query rows of one head as two slots of 128 (MMA M = 128) that
// share every K and V block of 128 keys.  Its blocks are those that some row
// sees: the first units' blocks, then the window's (WinBlocks); a slot skips
// the blocks that none of its own rows sees.  O = softmax(scale Q K^T) V with
// a running maximum and sum in float32, so the keys are read once.
//
// Bound by the tensor pipe and the exponential unit alike: a 128 x 128 block
// of a slot is 1024 clk of MMA (d = 128) and 16384 exponentials at 16 a clk.
// Two slots keep both busy: while the softmax of one slot works on its block,
// the tensor pipe runs the other's P V and next Q K^T.  Sharing K and V
// between the slots halves their way into shared memory, 32 bytes per MMA clk
// against the ~55 that TMA sustains here.
//
// Warps (384 threads): 0-3 softmax of slot 0, 4-7 of slot 1 (thread = row =
// TMEM lane), 8 loads Q and K, 9 loads V, 10 and 11 issue the MMAs of slot 0
// and 1 (an issuer each: a thread that has queued MMAs sees its next barrier
// test late).  TMEM: S0, S1 (128 columns each), O0, O1 (D each).  P, packed to
// 16 bits, overwrites the first half of its slot's S, 32 keys at a time, and is
// released to the P V MMAs in three parts; S of the slot's next block is
// queued right behind P V, so S_FULL also says that P V of the block before is
// complete and O may be rescaled (only when a row's maximum grew by more than
// 2^8).
//
// Left alone, the slots fall into step: both softmaxes at once, sharing the
// exponential unit, then both waiting for MMAs (3.4-3.7k clk for two 128 x 128
// blocks, 2048 of MMA).  So at d = 128 they take turns (window_wan5b 592 -> 540
// us; at d = 64, where the products are half as long, turns cost 4 %).
// window_wan5b, 6 heads of 27280 tokens, 8 frames and a sink: 540 us in bursts
// (1070 TFLOP/s, 66 % of the measured peak), 550-610 us under the power cap.
// Measured and not taken: a warpgroup on each half of a block's keys (four
// softmax warps a sub-partition, row maxima joined by an OR barrier) 8 %
// slower; 1/8 to 3/8 of the exponentials on the FMA pipe 2 to 10 % slower; the
// maximum before any exponential, P released in halves and the next S issued
// after a K wait 8 % slower; at d = 64 one slot a CTA and two CTAs an SM equal.
// Short windows at d = 64 (window_tokens, 165 us): of 38k clk a CTA 4.3k pass
// until the first scores, 2.5k a block, 1-2k more in each masked or first
// block, 4k from the last P to the end, 1.7k to the next CTA.
//
// Rounding: P is rounded to the 16-bit input type for the P V MMA (its sum l
// is taken from the float32 values), O once at the end.  fp16 is precise down to
// 2^-14 only, and a first unit that draws most of the weight leaves the others
// below that: its P and l carry 2^kWfUp, as far up as the rescale threshold
// allows (P <= 2^15; a first key e^14 above 8000 others, with V = 0: O off by
// 0.76 % without, 0.030 % with).
#pragma once

#include <cuda.h>

#include "window_args.cuh"
#include "window_ptx.cuh"

namespace vsa {

constexpr int kWfThreads = 384;
constexpr int kWfRows = 256;             // query rows a CTA
constexpr int kWfKeys = 128;             // keys a block
constexpr int kWfRegSoftmax = 208, kWfRegOther = 88;
static_assert(2 * 128 * kWfRegSoftmax + 128 * kWfRegOther <= kWfThreads * 168, "register split over the launch budget");
constexpr float kWfRescaleLog2 = 8.0f;
constexpr float kWfUp = 7.0f;            // fp16

template <int D>
struct WfSmem {
  static constexpr int kSlab = 128 * 128;              // 128 rows x 64 channels
  static constexpr int kSlabs = D / 64;
  static constexpr int kBuf = kSlabs * kSlab;          // 128 rows
  static constexpr int kKSt = 3, kVSt = 2;
  static constexpr int kQ = 0;                         // two slots; O leaves through them
  static constexpr int kK = 2 * kBuf;
  static constexpr int kV = kK + kKSt * kBuf;
  static constexpr int kBar = kV + kVSt * kBuf;
  static constexpr int kNumBars = 32;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kTotal = kMisc + 16 + 1024;     // 1024: alignment of the base
};

// P of a block is released in three parts: keys 0-63, 64-95, 96-127.
enum : int {
  WB_Q = 0, WB_S = 1 /* [slot] */, WB_P = 3 /* [slot][3] */, WB_O = 9 /* [slot] */, WB_DRAIN = 11,
  WB_K_FULL = 12, WB_K_EMPTY = 16, WB_V_FULL = 20, WB_V_EMPTY = 24
};

// Blocks of 128 keys that rows i0 .. i1 (inclusive) of a sequence see: ns
// first-unit blocks 0 .. ns-1, then w0 .. w1-1.  Keys outside [0, first) and
// [lo, hi) are seen by none of the rows.
struct WinBlocks {
  int first, lo, hi;
  int ns, w0, w1;
  __device__ __forceinline__ int count() const { return ns + w1 - w0; }
  __device__ __forceinline__ int block(int it) const { return it < ns ? it : w0 + it - ns; }
  __device__ __forceinline__ bool has(int blk) const { return blk < ns || (blk >= w0 && blk < w1); }
};

__device__ __forceinline__ WinBlocks win_blocks(const WinArgs& a, int len, int start, int i0, int i1) {
  WinBlocks w{0, 0, 0, 0, 0, 0};
  const int p1 = start + i1;
  if (p1 < 0 || i1 < i0) return w;
  const int p0 = max(start + i0, 0);
  const long long hi = min((p1 / a.unit + 1ll) * a.unit, static_cast<long long>(len));
  const long long lo = min(max((p0 / a.unit + 1ll - a.window) * a.unit, 0ll), hi);
  const long long first = min(a.sink_tok, hi);
  w.first = static_cast<int>(first);
  w.lo = static_cast<int>(lo);
  w.hi = static_cast<int>(hi);
  w.ns = (w.first + kWfKeys - 1) / kWfKeys;
  if (w.hi > w.lo) {
    w.w0 = w.lo / kWfKeys;
    w.w1 = (w.hi + kWfKeys - 1) / kWfKeys;
    w.ns = min(w.ns, w.w0);
  } else {
    w.w0 = w.w1 = w.ns;
  }
  return w;
}

// Mask of the 32 keys from c0 for one row.
__device__ __forceinline__ uint32_t vis_word(const RowVis& v, int c0) {
  return (low_bits(v.hi - c0) & ~low_bits(v.lo - c0)) | low_bits(v.first - c0);
}
// Mask words of the 128 keys from c0 for one row.
__device__ __forceinline__ void vis_words(const RowVis& v, int c0, uint32_t (&m)[4]) {
#pragma unroll
  for (int w = 0; w < 4; ++w) m[w] = vis_word(v, c0 + 32 * w);
}

// Zeros the rows of a 128-row tile (rows c0 .. of the keys or queries) outside
// [0, first) and [lo, hi): 128 threads, 8 lanes a row of 128 bytes (a thread a
// row would have all its stores in one bank: 3 us more for a CTA's one block).
template <int D>
__device__ __forceinline__ void zero_unseen(uint32_t buf, int c0, int first, int lo, int hi, int t) {
#pragma unroll
  for (int sl = 0; sl < D / 64; ++sl)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int row = 16 * e + t / 8, at = c0 + row;
      if (at >= first && (at < lo || at >= hi))
        st_shared_v4(buf + sl * WfSmem<D>::kSlab + row * 128u + (t % 8) * 16u, 0u, 0u, 0u, 0u);
    }
}

// splits > 1: blockIdx.z = batch * splits + split; a split takes its share of
// the CTA's blocks and writes its normalised O and its LSE to `part` in
// float32 ([split][B, Hq, Nq, D] and then [split][B, Hq, Nq]).
template <int D, bool F16>
__global__ void __launch_bounds__(kWfThreads, 1)
    window_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                      const __grid_constant__ WinArgs a, int splits, float* part) {
  using L = WfSmem<D>;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* sp = smem_raw + (base - raw);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sp + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sp + L::kMisc + 4);
  auto bar = [&](int id) -> uint32_t { return base + L::kBar + 8u * static_cast<uint32_t>(id); };

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int h = blockIdx.y, b = blockIdx.z / splits, split = blockIdx.z - b * splits;
  const int hk = h / a.group;
  // later rows first: with a long window they see the most keys
  const int i0 = (gridDim.x - 1 - blockIdx.x) * kWfRows;
  const int len = win_len(a, b), start = win_start(a, b, len);
  const WinBlocks wb = win_blocks(a, len, start, i0, min(i0 + kWfRows, a.Nq) - 1);
  const int n_all = wb.count();
  const int it0 = static_cast<int>(static_cast<long long>(n_all) * split / splits);
  const int n = static_cast<int>(static_cast<long long>(n_all) * (split + 1) / splits) - it0;   // this CTA's blocks

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kNumBars; ++i) {
      uint32_t cnt = 1;
      if (i >= WB_P && i < WB_P + 6) cnt = 128;
      if (i == WB_DRAIN || (i >= WB_K_EMPTY && i < WB_K_EMPTY + 4) || (i >= WB_V_EMPTY && i < WB_V_EMPTY + 4)) cnt = 2;
      mbar_init(bar(i), cnt);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 10) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 8) setmaxnreg_dec<kWfRegOther>();
  if (warp == 8 || warp == 9) {
    // ====================================================== TMA producers
    if (lane == 0) {
      const bool is_k = warp == 8;
      const CUtensorMap* tm = is_k ? &tmK : &tmV;
      const uint32_t buf0 = base + (is_k ? L::kK : L::kV);
      const int full = is_k ? WB_K_FULL : WB_V_FULL, empty = is_k ? WB_K_EMPTY : WB_V_EMPTY;
      const int stages = is_k ? L::kKSt : L::kVSt;
      if (is_k && n > 0) {
        mbar_arrive_expect_tx(bar(WB_Q), 2 * L::kBuf);
        for (int s = 0; s < 2; ++s)
          for (int sl = 0; sl < L::kSlabs; ++sl)
            tma_load_4d(base + L::kQ + s * L::kBuf + sl * L::kSlab, &tmQ, bar(WB_Q), sl * 64, i0 + 128 * s, h, b);
      }
      int st = 0, ph = 0, issued = 0;
      for (int j = 0; j < n; ++j) {
        if (j >= stages && !mbar_wait(bar(empty + st), ph ^ 1, abort_flag, a.err)) break;
        issued = j + 1;
        mbar_arrive_expect_tx(bar(full + st), L::kBuf);
        const int c0 = wb.block(it0 + j) * kWfKeys;
        for (int sl = 0; sl < L::kSlabs; ++sl)
          tma_load_4d(buf0 + st * L::kBuf + sl * L::kSlab, tm, bar(full + st), sl * 64, c0, hk, b);
        if (++st == stages) { st = 0; ph ^= 1; }
      }
      // let every issued copy land before the CTA can exit
      for (int j = max(0, issued - stages); j < issued; ++j)
        mbar_wait(bar(full + j % stages), (j / stages) & 1, nullptr, a.err);
      if (is_k && n > 0) mbar_wait(bar(WB_Q), 0, nullptr, a.err);
    }
    __syncwarp();
  } else if (warp >= 10) {
    // ====================================================== MMA issuers
    const int s = warp - 10;
    const WinBlocks mine = win_blocks(a, len, start, i0 + 128 * s, min(i0 + 128 * s + 128, a.Nq) - 1);
    constexpr uint32_t idS = idesc_f16kind_f32(128, kWfKeys, false, F16);
    constexpr uint32_t idPV = idesc_f16kind_f32(128, D, true, F16);
    const uint32_t tS = tmem + 128u * s, tO = tmem + 256u + D * s;
    const uint32_t sQ = base + L::kQ + s * L::kBuf;
    bool ok = n == 0 || __all_sync(0xffffffffu, mbar_wait(bar(WB_Q), 0, abort_flag, a.err));
    // Blocks that this slot does not use are released as they arrive, K and V
    // together (waiting for each keeps an issuer from running ahead a phase).
    auto skip = [&](int j) {
      while (ok && j < n && !mine.has(wb.block(it0 + j))) {
        const int ks = j % L::kKSt, vs = j % L::kVSt;
        ok = __all_sync(0xffffffffu, mbar_wait(bar(WB_K_FULL + ks), (j / L::kKSt) & 1, abort_flag, a.err) &&
                                         mbar_wait(bar(WB_V_FULL + vs), (j / L::kVSt) & 1, abort_flag, a.err));
        if (ok && lane == 0) {
          mbar_arrive(bar(WB_K_EMPTY + ks));
          mbar_arrive(bar(WB_V_EMPTY + vs));
        }
        ++j;
      }
      return j;
    };
    auto wait_k = [&](int j) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar(WB_K_FULL + j % L::kKSt), (j / L::kKSt) & 1, abort_flag, a.err));
    };
    // (elected lane) S of block j over the slot's score columns
    auto scores = [&](int j) {
      const int ks = j % L::kKSt;
      const uint32_t kb = base + L::kK + ks * L::kBuf;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const int off = (kk / 4) * L::kSlab + (kk % 4) * 32;
        mma_ss(tS, smem_desc_sw128(sQ + off, 16, 1024), smem_desc_sw128(kb + off, 16, 1024), idS, kk > 0 ? 1u : 0u);
      }
      mma_commit(bar(WB_S + s));
      mma_commit(bar(WB_K_EMPTY + ks));
    };
    int j = skip(0), c = 0;
    if (ok && j < n) {
      wait_k(j);
      if (ok) {
        tc_fence_after();
        if (elect_one_sync()) scores(j);
        __syncwarp();
      }
    }
    while (ok && j < n) {
      const int vs = j % L::kVSt;
      const uint32_t vb = base + L::kV + vs * L::kBuf;
      // S of the next block is queued right behind this block's last P V: its
      // K is waited for before, since a thread's barrier test behind queued
      // MMAs waits for them to drain.  Not across blocks that are skipped
      // (their V stage may be this block's, which is not released yet).
      const bool next = j + 1 < n && mine.has(wb.block(it0 + j + 1));
      ok = __all_sync(0xffffffffu, mbar_wait(bar(WB_V_FULL + vs), (j / L::kVSt) & 1, abort_flag, a.err));
#pragma unroll
      for (int pt = 0; pt < 3 && ok; ++pt) {
        if (pt == 1 && next) wait_k(j + 1);
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(WB_P + 3 * s + pt), c & 1, abort_flag, a.err));
        if (!ok) break;
        tc_fence_after();
        if (elect_one_sync()) {
#pragma unroll
          for (int kk = pt == 0 ? 0 : 2 + 2 * pt; kk < 4 + 2 * pt; ++kk)    // 16 keys = 16 rows of 128 bytes
            mma_ts(tO, tS + 8u * kk, smem_desc_sw128(vb + kk * 2048, L::kSlab, 1024), idPV,
                   (c > 0 || kk > 0) ? 1u : 0u);
          if (pt == 2) {
            if (next) scores(j + 1);
            mma_commit(bar(WB_V_EMPTY + vs));
          }
        }
        __syncwarp();
      }
      ++c;
      if (!ok) break;
      if (next) {
        ++j;
        continue;
      }
      j = skip(j + 1);
      if (ok && j < n) {
        wait_k(j);
        if (!ok) break;
        tc_fence_after();
        if (elect_one_sync()) scores(j);
        __syncwarp();
      }
    }
    if (elect_one_sync()) {
      if (c > 0) mma_commit(bar(WB_O + s));
      mma_commit(bar(WB_DRAIN));
    }
    __syncwarp();
    mbar_wait(bar(WB_DRAIN), 0, nullptr, a.err);     // every MMA has finished before TMEM is freed
  } else {
    // ====================================================== softmax
    setmaxnreg_inc<kWfRegSoftmax>();
    const int s = warp / 4, r = threadIdx.x % 128;
    const int i = i0 + 128 * s + r;
    const uint32_t lane_base = static_cast<uint32_t>((warp % 4) * 32) << 16;
    const uint32_t tS = tmem + lane_base + 128u * s, tO = tmem + lane_base + 256u + D * s;
    const WinBlocks mine = win_blocks(a, len, start, i0 + 128 * s, min(i0 + 128 * s + 128, a.Nq) - 1);
    RowVis vis{0, 0, 0};
    if (i < a.Nq) vis = row_vis(a, len, start + i);
    constexpr float kUp = F16 ? kWfUp : 0.f;
    float m = -INFINITY, l = 0.f;
    int c = 0;
    // After a wait that gave up (ok = false) the loop goes on without waiting, so
    // that both slots meet at every hand-over.
    bool ok = true;
    // The slots take turns: slot 0's exponentials of a block, then slot 1's, and
    // so on (named barriers 3 and 4, a turn a block whether the slot uses it or
    // not); the turn is passed on after half of them.
    constexpr bool kTurns = D == 128;
    if (kTurns && s == 1 && n > 0) named_bar_arrive(3, 256);
    const uint64_t sc2 = f2_pack(a.scale_log2, a.scale_log2);
    for (int j = 0; j < n; ++j) {
      const int blk = wb.block(it0 + j), c0 = blk * kWfKeys;
      const bool pass = s == 0 || j < n - 1;           // (slot 0 waits once less than slot 1 has turns)
      if (!mine.has(blk)) {
        if (kTurns) {
          named_bar_sync(3 + s, 256);
          if (pass) named_bar_arrive(4 - s, 256);
        }
        continue;
      }
      const bool row_full = i >= a.Nq || c0 + kWfKeys <= vis.first || (c0 >= vis.lo && c0 + kWfKeys <= vis.hi);
      const bool masked = __any_sync(0xffffffffu, !row_full);
      // Keys of the block that no row of the CTA sees may hold anything: zero
      // their V rows (0 * NaN would reach O).  Both slots write the same zeros.
      if ((c0 + kWfKeys > wb.hi || c0 < wb.lo) && c0 + kWfKeys > wb.first) {
        const int vs = j % L::kVSt;
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(WB_V_FULL + vs), (j / L::kVSt) & 1, abort_flag, a.err));
        zero_unseen<D>(base + L::kV + vs * L::kBuf, c0, wb.first, wb.lo, wb.hi, r);
        fence_proxy_async_smem();
      }
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(WB_S + s), c & 1, abort_flag, a.err));
      tc_fence_after();
      uint32_t x[128];
      tmem_ld32(tS + 0, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
      tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&x[32]));
      tmem_ld32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(&x[64]));
      tmem_ld32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(&x[96]));
      tmem_wait_ld();
      sched_fence(a);
      if (masked) {
        uint32_t mw[4];
        vis_words(vis, c0, mw);
#pragma unroll
        for (int e = 0; e < 128; ++e)
          if (!((mw[e >> 5] >> (e & 31)) & 1u)) x[e] = __float_as_uint(-INFINITY);
      }
      float mx4[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) mx4[e] = __uint_as_float(x[e]);
#pragma unroll
      for (int e = 4; e < 128; e += 2)
        mx4[(e >> 1) & 3] = fmax3(mx4[(e >> 1) & 3], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
      // P of the first 32 keys against the reference as it stands, made while
      // the maximum is; kept unless the maximum moves the reference.
      uint64_t ls2[4] = {0ull, 0ull, 0ull, 0ull};
      auto expo = [&](int at, uint64_t nm2, uint32_t* pk) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint64_t z2 = f2_fma(f2_pack(__uint_as_float(x[at + 2 * e]), __uint_as_float(x[at + 2 * e + 1])), sc2, nm2);
          float z0, z1;
          f2_unpack(z2, z0, z1);
          const float p0 = ex2_approx(z0), p1 = ex2_approx(z1);
          ls2[e & 3] = f2_add(ls2[e & 3], f2_pack(p0, p1));
          pk[e] = pack_elem2<F16>(p0, p1);
        }
      };
      uint32_t pk[16];
      float mu = m == -INFINITY ? 0.f : m;
      if (kTurns) named_bar_sync(3 + s, 256);
      expo(0, f2_pack(kUp - mu, kUp - mu), pk);
      const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * a.scale_log2;
      sched_fence(a);
      if (__any_sync(0xffffffffu, mx > m + kWfRescaleLog2)) {
        const float m_new = mx > m + kWfRescaleLog2 ? mx : m;
        const float f = m_new == m ? 1.f : (m == -INFINITY ? 0.f : ex2_approx(m - m_new));
        l *= f;
        m = m_new;
        if (c > 0) {
          // P V of the slot's block before is complete (S_FULL), so O is still
#pragma unroll
          for (int q = 0; q < D / 16; ++q) {
            uint32_t ov[16];
            tmem_ld16(tO + 16u * q, ov);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f);
            tmem_st16(tO + 16u * q, ov);
          }
        }
        mu = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int e = 0; e < 4; ++e) ls2[e] = 0ull;
        expo(0, f2_pack(kUp - mu, kUp - mu), pk);
      }
      const uint64_t nm2 = f2_pack(kUp - mu, kUp - mu);
      sched_fence(a);
      tmem_st16(tS, pk);
#pragma unroll
      for (int q = 1; q < 4; ++q) {
        expo(32 * q, nm2, pk);
        if (kTurns && q == 1 && pass) named_bar_arrive(4 - s, 256);
        tmem_st16(tS + 16u * q, pk);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(WB_P + 3 * s + q - 1));
        sched_fence(a);
      }
      float s0, s1;
      f2_unpack(f2_add(f2_add(ls2[0], ls2[1]), f2_add(ls2[2], ls2[3])), s0, s1);
      l += s0 + s1;
      ++c;
    }

    // ---- epilogue: O / l, staged in the slot's Q buffer (every MMA that read
    // Q is complete by O_FULL) with the 128-byte swizzle of the boxes, one TMA
    // store a slab; rows past Nq are dropped by the map
    if (ok && n > 0)       // (a slot without blocks: Q has landed, so that it cannot overwrite the staged zeros)
      ok = __all_sync(0xffffffffu, mbar_wait(bar(c > 0 ? WB_O + s : WB_Q), 0, abort_flag, a.err));
    tc_fence_after();
    // (l = 0: the row sees nothing; a NaN among what it sees stays one)
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const float lse = l == 0.f ? -INFINITY : (m - kUp + log2f(l)) * 0.69314718055994530942f;
    const size_t row = (static_cast<size_t>(b) * a.Hq + h) * a.Nq + i;
    const size_t rows = static_cast<size_t>(a.B) * a.Hq * a.Nq;
    if (n > 0 && splits == 1) {
      if (ok) {
        const uint32_t orow = base + L::kQ + s * L::kBuf + r * 128u;
#pragma unroll
        for (int q4 = 0; q4 < D / 32; ++q4) {
          uint32_t ov[32];
          if (c > 0) {
            tmem_ld32(tO + 32u * q4, ov);
            tmem_wait_ld();
          }
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            pk[e] = l == 0.f ? 0u : pack_elem2<F16>(__uint_as_float(ov[2 * e]) * inv, __uint_as_float(ov[2 * e + 1]) * inv);
          const uint32_t at = orow + (q4 >> 1) * L::kSlab;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            st_shared_v4(at + static_cast<uint32_t>(((q4 & 1) * 4 + e) ^ (r & 7)) * 16u, pk[4 * e], pk[4 * e + 1],
                         pk[4 * e + 2], pk[4 * e + 3]);
        }
        fence_proxy_async_smem();
      }
      named_bar_sync(1 + s, 128);
      if (ok && r == 0 && i0 + 128 * s < a.Nq) {
        for (int sl = 0; sl < L::kSlabs; ++sl)
          tma_store_4d(&tmO, base + L::kQ + s * L::kBuf + sl * L::kSlab, sl * 64, i0 + 128 * s, h, b);
        bulk_commit_group();
        bulk_wait_group_read0();
      }
      if (ok && i < a.Nq) a.lse[row] = lse;
    } else if (ok && splits == 1) {
      // no row of the CTA sees anything
      if (i < a.Nq) {
        uint4* o = reinterpret_cast<uint4*>(a.out + b * a.os[0] + i * a.os[1] + h * a.os[2]);
#pragma unroll
        for (int e = 0; e < D / 8; ++e) o[e] = make_uint4(0u, 0u, 0u, 0u);
        a.lse[row] = -INFINITY;
      }
    } else if (ok) {
      float* op = part + (split * rows + row) * D;
#pragma unroll
      for (int q4 = 0; q4 < D / 32; ++q4) {
        uint32_t ov[32];
        if (c > 0) {
          tmem_ld32(tO + 32u * q4, ov);
          tmem_wait_ld();
        }
        if (i < a.Nq) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
            if (l != 0.f)
              f = make_float4(__uint_as_float(ov[4 * e]) * inv, __uint_as_float(ov[4 * e + 1]) * inv,
                              __uint_as_float(ov[4 * e + 2]) * inv, __uint_as_float(ov[4 * e + 3]) * inv);
            reinterpret_cast<float4*>(op + 32 * q4)[e] = f;
          }
        }
      }
      if (i < a.Nq) part[splits * rows * D + split * rows + row] = lse;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 10) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// O = sum_s e^(lse_s - L) O_s, L = log sum_s e^lse_s over the splits of a row:
// a CTA a row, its eight warps every eighth split (there are few rows here, and
// up to hundreds of splits), D / 32 channels a lane; reads what the splits
// wrote once.
template <int D, bool F16>
__global__ void __launch_bounds__(256) window_combine_kernel(const __grid_constant__ WinArgs a, int splits, const float* part) {
  constexpr int W = 8;
  __shared__ float so[W][D];
  __shared__ float sw[W];
  const size_t rows = static_cast<size_t>(a.B) * a.Hq * a.Nq, row = blockIdx.x;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const float* ls = part + splits * rows * D + row;
  float mx = -INFINITY;
  for (int s = lane; s < splits; s += 32) mx = fmaxf(mx, ls[s * rows]);
#pragma unroll
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (mx == -INFINITY) mx = 0.f;                        // (no split sees anything, or one holds a NaN)
  float acc[D / 32] = {}, sum = 0.f;
#pragma unroll 4
  for (int s = warp; s < splits; s += W) {
    const float w = exp2f((ls[s * rows] - mx) * 1.4426950408889634f);
    sum += w;
    const float* op = part + (s * rows + row) * D + lane;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] = fmaf(w, op[32 * e], acc[e]);
  }
#pragma unroll
  for (int e = 0; e < D / 32; ++e) so[warp][lane + 32 * e] = acc[e];
  if (lane == 0) sw[warp] = sum;
  __syncthreads();
  if (threadIdx.x >= D / 2) return;
  sum = 0.f;
  float x = 0.f, y = 0.f;
#pragma unroll
  for (int k = 0; k < W; ++k) {
    sum += sw[k];
    x += so[k][2 * threadIdx.x];
    y += so[k][2 * threadIdx.x + 1];
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int i = static_cast<int>(row % a.Nq);
  const size_t bh = row / a.Nq;
  const int h = static_cast<int>(bh % a.Hq), b = static_cast<int>(bh / a.Hq);
  reinterpret_cast<uint32_t*>(a.out + b * a.os[0] + i * a.os[1] + h * a.os[2])[threadIdx.x] =
      pack_elem2<F16>(x * inv, y * inv);
  if (threadIdx.x == 0) a.lse[row] = sum == 0.f ? -INFINITY : mx + logf(sum);
}

}  // namespace vsa

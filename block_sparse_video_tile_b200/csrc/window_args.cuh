// window_args.cuh -- which keys a query of vsa_window_attn sees, evaluated the
// same way by every kernel of the call and its gradient.
//
// With units of `unit` tokens, the keys that position p sees are two ranges,
// [0, first) (the first units) and [lo, hi) (the window), both bounded by the
// sequence's length: hi = end of p's unit, lo = start of the unit window - 1
// before it, first = end of unit sink - 1.  All three grow with p, so the
// keys that a block of rows sees are bounded by its first and last row.
#pragma once

#include <cstdint>

namespace vsa {

struct WinArgs {
  int B, Hq, Hkv, group;     // group = Hq / Hkv query heads read one key/value head
  int Nq, Nk;
  int unit, window;          // tokens a unit; units a query looks back, its own included
  long long sink_tok;        // tokens of the first units
  const int32_t* kv_len;     // [B] or nullptr
  const int32_t* q_start;    // [B] or nullptr
  const uint16_t *q, *k, *v, *o, *d_o;
  uint16_t *out, *dq, *dk, *dv;
  float *lse, *delta;        // [B, Hq, Nq]
  long long qs[3], ks[3], vs[3], os[3], dos[3], dqs[3], dks[3], dvs[3];   // (b, n, h) strides, elements
  float scale, scale_log2;   // softmax_scale, softmax_scale * log2(e)
  // fp16 gradient: [B, Hkv] largest bound on |dP - delta| (float bits), and
  // [B, Hkv, chunks] largest |V_j|^2
  unsigned int* grad_bound;
  float* v_norms;
  int chunks;
  unsigned int* err;
};

constexpr int kWinMaxPos = 1 << 30;        // of q_start; start + row stays below 2^31
constexpr int kWinMaxRows = (1 << 30) - 512;

__device__ __forceinline__ int win_len(const WinArgs& a, int b) {
  return a.kv_len == nullptr ? a.Nk : min(max(__ldg(a.kv_len + b), 0), a.Nk);
}
__device__ __forceinline__ int win_start(const WinArgs& a, int b, int len) {
  return a.q_start == nullptr ? len - a.Nq : min(max(__ldg(a.q_start + b), -kWinMaxPos), kWinMaxPos);
}

// Position p sees [0, first) and [lo, hi); first <= lo (touching ranges are
// joined into [0, hi) with first = 0); nothing: first = 0 and lo = hi (0 before
// position 0, the length where the window begins behind the last key).
struct RowVis {
  int first, lo, hi;
  __device__ __forceinline__ bool sees(int j) const { return j < hi && (j >= lo || j < first); }
};

__device__ __forceinline__ RowVis row_vis(const WinArgs& a, int len, int p) {
  RowVis r{0, 0, 0};
  if (p < 0) return r;
  const int u = p / a.unit;
  const long long hi = min((u + 1ll) * a.unit, static_cast<long long>(len));
  const long long lo = min(max((u + 1ll - a.window) * a.unit, 0ll), hi);
  const long long first = min(a.sink_tok, hi);
  r.hi = static_cast<int>(hi);
  if (first >= lo) return r;                       // (first = lo = 0)
  r.lo = static_cast<int>(lo);
  r.first = static_cast<int>(first);
  return r;
}

// The query rows [lo, hi) that see a key; nobody: lo >= hi.
struct KeyVis {
  int lo, hi;
};

__device__ __forceinline__ KeyVis key_vis(const WinArgs& a, int len, int start, int key) {
  if (key >= len) return KeyVis{0, 0};
  const long long u = key / a.unit, p0 = u * a.unit;
  const long long p1 = key < a.sink_tok ? (1ll << 40) : (u + a.window) * a.unit;
  const long long Nq = a.Nq;
  return KeyVis{static_cast<int>(min(max(p0 - start, 0ll), Nq)), static_cast<int>(min(max(p1 - start, 0ll), Nq))};
}

}  // namespace vsa

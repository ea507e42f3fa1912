// window.cu -- vsa_window_attn and its gradient: argument checks and launches
// (declared in include/vsa.h).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "vsa.h"
#include "tma_encode.cuh"
#include "vsa_host.h"
#include "window_args.cuh"
#include "window_bwd.cuh"
#include "window_fwd.cuh"
#include "window_step.cuh"

namespace vsa {

static int win_args(const vsa_window* w, float scale, WinArgs* a) {
  if (w == nullptr) return VSA_ERR_INVALID_ARG;
  if (w->B <= 0 || w->Hq <= 0 || w->Hkv <= 0 || w->Nq <= 0 || w->Nk <= 0) return VSA_ERR_INVALID_ARG;
  if (w->Hq % w->Hkv != 0 || w->window < 1 || w->sink < 0 || w->unit < 1) return VSA_ERR_INVALID_ARG;
  if (w->d != 64 && w->d != 128) return VSA_ERR_UNSUPPORTED;
  if (w->dtype != VSA_DTYPE_BF16 && w->dtype != VSA_DTYPE_F16) return VSA_ERR_UNSUPPORTED;
  if (!(scale > 0.f) || !std::isfinite(scale)) return VSA_ERR_INVALID_ARG;
  if (!aligned_to(w->kv_len, 4) || !aligned_to(w->q_start, 4)) return VSA_ERR_ALIGNMENT;
  if (w->Nq > kWinMaxRows || w->Nk > kWinMaxRows || w->B > 65535 || w->Hq > 65535) return VSA_ERR_TOO_LARGE;
  a->B = w->B; a->Hq = w->Hq; a->Hkv = w->Hkv; a->group = w->Hq / w->Hkv;
  a->Nq = w->Nq; a->Nk = w->Nk;
  a->unit = w->unit;
  a->window = w->window;
  a->sink_tok = 1ll * w->sink * w->unit;
  a->kv_len = w->kv_len;
  a->q_start = w->q_start;
  a->scale = scale;
  a->scale_log2 = scale * 1.4426950408889634f;
  int rc;
  if ((rc = take_strides(w->q_s, w->B, w->Nq, w->Hq, w->d, a->qs)) != VSA_OK ||
      (rc = take_strides(w->k_s, w->B, w->Nk, w->Hkv, w->d, a->ks)) != VSA_OK ||
      (rc = take_strides(w->v_s, w->B, w->Nk, w->Hkv, w->d, a->vs)) != VSA_OK ||
      (rc = take_strides(w->o_s, w->B, w->Nq, w->Hq, w->d, a->os)) != VSA_OK)
    return rc;
  return VSA_OK;
}

static int win_bwd_strides(const vsa_window* w, WinArgs* a) {
  int rc;
  if ((rc = take_strides(w->do_s, w->B, w->Nq, w->Hq, w->d, a->dos)) != VSA_OK ||
      (rc = take_strides(w->dq_s, w->B, w->Nq, w->Hq, w->d, a->dqs)) != VSA_OK ||
      (rc = take_strides(w->dk_s, w->B, w->Nk, w->Hkv, w->d, a->dks)) != VSA_OK ||
      (rc = take_strides(w->dv_s, w->B, w->Nk, w->Hkv, w->d, a->dvs)) != VSA_OK)
    return rc;
  return VSA_OK;
}

// A strided head tensor as (d, N, H, B) with boxes of 64 channels x `rows`
// rows of one head; reads past N give zeros, writes past N are dropped.
static int encode_heads(CUtensorMap* m, const void* ptr, int B, int N, int H, int d, const long long s[3], int rows,
                        bool f16) {
  EncodeTiledFn fn = get_encode_fn();
  if (fn == nullptr) return VSA_ERR_CUDA;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(H),
                        static_cast<cuuint64_t>(B)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(s[1]) * 2, static_cast<cuuint64_t>(s[2]) * 2,
                           static_cast<cuuint64_t>(s[0]) * 2};
  cuuint32_t box[4] = {64u, static_cast<cuuint32_t>(rows), 1u, 1u};
  cuuint32_t es[4] = {1, 1, 1, 1};
  const CUresult r = fn(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                        const_cast<void*>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? VSA_OK : VSA_ERR_CUDA;
}

// How a forward call is run: few rows a key/value head take the step kernel,
// others the tcgen05 kernel (which gives each query head of a group CTAs of its
// own, however few its rows); either splits its keys when its CTAs are too few,
// as far as the most keys that a row can see allow (the lengths are on the
// device).  Where the two cross depends on the group; us of the step and of the
// tcgen05 kernel, 16384 keys, d = 128:
//   rows a key/value head     16        32        48        64        80        96
//   2 x 8 heads, group 4    54 126    71 126    91 128    90 128   131 130   148 130
//   8 x 8 heads, group 4   115 449   152 449   262 451   277 451   375 448   459 451
//   2 x 8 heads, group 1    54  46    71  46    91  48    90  48   131  50   148  50
//   2 x 24 heads, group 1  118  95   148  97   205  99   262 101   277 105   277 108
// kWsMaxRows suits groups of 4 and more; it is late for a group of 1.
constexpr int kWsMaxRows = 64;
constexpr int kWfFixed = 6;              // what a CTA of the tcgen05 kernel costs besides its blocks, in blocks
// CTAs that a step call asks for, two an SM: with splits joined in a cluster 1.5
// rounds of them (64 row tiles of 16384 keys: 5 splits 127 us, 7 95 us, 8 90 us,
// 18 and a second kernel 104 us; 256 tiles of 2048: 2 splits 51 us, 8 84 us), with
// the second kernel one round (8 tiles of 65536: 51 us, two rounds 56 us).
// Between them, where 1.5 rounds ask for 9 to 12 splits, a round and the second
// kernel against 8 joined splits (32768 keys): 37 tiles 130 and 168 us, 40 tiles
// 179 and 172, 48 tiles 202 and 174, 55 tiles 230 and 184.
constexpr int kWsClusterCtas = 148 * 3, kWsSplitCtas = 148 * 2;

struct WinPlan {
  bool step, cluster;        // cluster: the splits are joined by the kernel itself
  int splits;
  int partial() const { return cluster ? 1 : splits; }      // splits that leave partial results
};

static WinPlan win_plan(const WinArgs& a) {
  WinPlan p;
  const long long rows = 1ll * a.Nq * a.group;
  p.step = rows <= kWsMaxRows && a.Hkv * ((rows + kWsRows - 1) / kWsRows) <= 65535;      // (grid.y)
  // the most keys that `span` consecutive queries see
  auto keys_of = [&](long long span) {
    return std::min<long long>(
        a.Nk, std::min(a.sink_tok, 1ll << 32) + std::min((a.window + 1ll) * a.unit, 1ll << 32) + span);
  };
  if (p.step) {
    const long long ctas = 1ll * a.B * a.Hkv * ((rows + kWsRows - 1) / kWsRows);
    const long long most = std::max(1ll, keys_of(a.Nq) / (kWsKeys * kWsWarps * 2));   // two tiles a warp at least
    long long want = std::min((kWsClusterCtas + ctas - 1) / ctas, most);
    p.cluster = want <= kWsCluster;
    // one split more if it leaves less of the last round of CTAs empty
    auto used = [&](long long s) { return 1.0 * ctas * s / (148 * 2 * ((ctas * s + 295) / 296)); };
    if (want < kWsCluster && want < most && used(want + 1) > used(want)) ++want;
    p.splits = static_cast<int>(std::max(1ll, p.cluster ? want : std::min({(kWsSplitCtas + ctas - 1) / ctas, most, 256ll})));
    if (p.splits == 1) p.cluster = false;
  } else {
    // Splits s that make rounds * (blocks of a split + kWfFixed) least: the rounds
    // of CTAs that the SMs take, and what starting and ending a CTA costs in
    // blocks' time (about 10k clk of ~1.7k).  Writing and reading partial results
    // comes on top, so a split has to save a fifth (24 heads, 880 queries, 94
    // blocks: 209 us in one round of 96 CTAs, 232 us as three splits in two; 6
    // heads, 160 blocks: 271 us, 82 us with 6 splits).
    p.cluster = false;
    p.splits = 1;
    const long long ctas = 1ll * ((a.Nq + kWfRows - 1) / kWfRows) * a.Hq * a.B;
    const long long blocks = (keys_of(kWfRows) + kWfKeys - 1) / kWfKeys;
    long long best = (ctas + 147) / 148 * (blocks + kWfFixed) * 4 / 5;
    for (long long s = 2; s <= 8 && s * 4 <= blocks && a.B * s <= 65535; ++s) {
      const long long cost = (ctas * s + 147) / 148 * ((blocks + s - 1) / s + kWfFixed) + kWfFixed;
      if (cost < best) {
        best = cost;
        p.splits = static_cast<int>(s);
      }
    }
  }
  return p;
}

static size_t win_fwd_bytes(const WinArgs& a, int d, int splits) {
  return splits == 1 ? 0 : static_cast<size_t>(splits) * a.B * a.Hq * a.Nq * (d + 1) * sizeof(float);
}

template <int D, bool F16>
static int launch_combine(const WinArgs& a, int splits, const float* part, cudaStream_t st) {
  if (splits == 1) return VSA_OK;
  const long long rows = 1ll * a.B * a.Hq * a.Nq;
  window_combine_kernel<D, F16><<<static_cast<unsigned>(rows), 256, 0, st>>>(a, splits, part);
  return cudaGetLastError() == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
}

template <int D, bool F16, bool CLUSTER>
static int launch_step_as(const WinArgs& a, int splits, float* part, cudaStream_t st) {
  constexpr int smem = WsSmem<D>::kTotal;
  if (cudaFuncSetAttribute(window_step_kernel<D, F16, CLUSTER>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
      cudaSuccess)
    return VSA_ERR_CUDA;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(splits, a.Hkv * ((a.Nq * a.group + kWsRows - 1) / kWsRows), a.B);
  cfg.blockDim = dim3(kWsThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = CLUSTER ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, window_step_kernel<D, F16, CLUSTER>, a, splits, part) != cudaSuccess) return VSA_ERR_CUDA;
  return CLUSTER ? VSA_OK : launch_combine<D, F16>(a, splits, part, st);
}

template <int D, bool F16>
static int launch_fwd(const WinArgs& a, int splits, float* part, cudaStream_t st) {
  CUtensorMap mq, mk, mv, mo;
  int rc;
  if ((rc = encode_heads(&mq, a.q, a.B, a.Nq, a.Hq, D, a.qs, 128, F16)) != VSA_OK ||
      (rc = encode_heads(&mk, a.k, a.B, a.Nk, a.Hkv, D, a.ks, kWfKeys, F16)) != VSA_OK ||
      (rc = encode_heads(&mv, a.v, a.B, a.Nk, a.Hkv, D, a.vs, kWfKeys, F16)) != VSA_OK ||
      (rc = encode_heads(&mo, a.out, a.B, a.Nq, a.Hq, D, a.os, 128, F16)) != VSA_OK)
    return rc;
  if (cudaFuncSetAttribute(window_fwd_kernel<D, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           WfSmem<D>::kTotal) != cudaSuccess)
    return VSA_ERR_CUDA;
  const dim3 grid((a.Nq + kWfRows - 1) / kWfRows, a.Hq, a.B * splits);
  window_fwd_kernel<D, F16><<<grid, kWfThreads, WfSmem<D>::kTotal, st>>>(mq, mk, mv, mo, a, splits, part);
  if (cudaGetLastError() != cudaSuccess) return VSA_ERR_CUDA;
  return launch_combine<D, F16>(a, splits, part, st);
}

template <int D, bool F16>
static int launch_any(const WinArgs& a, const WinPlan& p, float* part, cudaStream_t st) {
  if (!p.step) return launch_fwd<D, F16>(a, p.splits, part, st);
  return p.cluster ? launch_step_as<D, F16, true>(a, p.splits, part, st) : launch_step_as<D, F16, false>(a, p.splits, part, st);
}

// Key blocks are shared among CTAs when one would walk much longer than an
// SM's share of all the walks (kWbShares shares an SM), but no CTA walks fewer
// than about kWbLeast blocks for it (setting one up costs as much as walking
// several).  Walks are bounded from above: the lengths are on the device.
constexpr int kWbShares = 2, kWbLeast = 12, kWbMost = 32;

static DkvSplit dkv_split(const WinArgs& a) {
  DkvSplit s;
  s.blocks = (a.Nk + kWbRows - 1) / kWbRows;
  s.heavy = static_cast<int>(std::min<long long>(s.blocks, (a.sink_tok + kWbRows - 1) / kWbRows));
  const long long all = (a.Nq + kWbRows - 1) / kWbRows;
  const long long seen = std::min(all, (std::min(1ll * a.window * a.unit, 1ll << 32) + a.unit + kWbRows) / kWbRows + 1);
  const long long wh = all * a.group, wn = seen * a.group;             // blocks that a key block is walked with
  // (in 64-bit floats: the product of the largest extents passes 63 bits)
  const double sum = (1.0 * s.heavy * wh + 1.0 * (s.blocks - s.heavy) * wn) * a.B * a.Hkv;
  const double share = std::max<double>(kWbLeast, std::ceil(sum / (148 * kWbShares)));
  auto parts = [&](long long walk) { return static_cast<int>(std::min<double>(kWbMost, std::max(1.0, std::ceil(walk / share)))); };
  s.sh = parts(wh);
  s.sn = parts(wn);                                    // (wn <= wh: sn <= sh)
  return s;
}

// delta, fp16's bounds, then the partial tiles of shared key blocks
static size_t win_delta_bytes(const vsa_window* w) {
  return (static_cast<size_t>(w->B) * w->Hq * w->Nq * sizeof(float) + 255) & ~static_cast<size_t>(255);
}
// fp16: the bounds and norms of WinArgs::grad_bound and v_norms
static int win_chunks(const vsa_window* w) { return std::min(128, (w->Nk + 127) / 128); }
static size_t win_range_bytes(const vsa_window* w) {
  if (w->dtype != VSA_DTYPE_F16) return 0;
  return (static_cast<size_t>(w->B) * w->Hkv * (1 + win_chunks(w)) * sizeof(float) + 255) & ~static_cast<size_t>(255);
}
static size_t win_bwd_bytes(const vsa_window* w, const DkvSplit& s) {
  return win_delta_bytes(w) + win_range_bytes(w) + static_cast<size_t>(w->B) * w->Hkv * s.tiles() * (2 * 128 * sizeof(float)) * w->d;
}

// For fp16 the keys' norms, then dQ (which also writes delta), then dK and dV.
template <int D, bool F16>
static int launch_bwd(const WinArgs& a, const DkvSplit& ds, float* part, cudaStream_t st) {
  CUtensorMap mq, mg, mk, mv, mdq, mdk, mdv;
  int rc;
  if ((rc = encode_heads(&mq, a.q, a.B, a.Nq, a.Hq, D, a.qs, kWbRows, F16)) != VSA_OK ||
      (rc = encode_heads(&mg, a.d_o, a.B, a.Nq, a.Hq, D, a.dos, kWbRows, F16)) != VSA_OK ||
      (rc = encode_heads(&mk, a.k, a.B, a.Nk, a.Hkv, D, a.ks, kWbRows, F16)) != VSA_OK ||
      (rc = encode_heads(&mv, a.v, a.B, a.Nk, a.Hkv, D, a.vs, kWbRows, F16)) != VSA_OK ||
      (rc = encode_heads(&mdq, a.dq, a.B, a.Nq, a.Hq, D, a.dqs, kWbRows, F16)) != VSA_OK ||
      (rc = encode_heads(&mdk, a.dk, a.B, a.Nk, a.Hkv, D, a.dks, kWbRows, F16)) != VSA_OK ||
      (rc = encode_heads(&mdv, a.dv, a.B, a.Nk, a.Hkv, D, a.dvs, kWbRows, F16)) != VSA_OK)
    return rc;
  constexpr int smem = WbSmem<D>::kTotal;
  if (cudaFuncSetAttribute(window_dq_kernel<D, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      cudaFuncSetAttribute(window_dkv_kernel<D, F16, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
          cudaSuccess ||
      cudaFuncSetAttribute(window_dkv_kernel<D, F16, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
          cudaSuccess)
    return VSA_ERR_CUDA;
  if (F16) {
    window_v_norm_kernel<D><<<dim3(a.chunks, a.Hkv, a.B), 256, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return VSA_ERR_CUDA;
  }
  // fp16: the dQ kernel is set up while the norms are made, and waits for them
  // itself (window_bwd_tokens 148.5 -> 145.0 us)
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.Nq + kWbRows - 1) / kWbRows, a.Hq, a.B);
  cfg.blockDim = dim3(kWbThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = F16 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, window_dq_kernel<D, F16>, mq, mg, mk, mv, mdq, a) != cudaSuccess) return VSA_ERR_CUDA;
  const dim3 grid(ds.ctas(), a.Hkv, a.B);
  if (ds.tiles() > 0)
    window_dkv_kernel<D, F16, true><<<grid, kWbThreads, smem, st>>>(mq, mg, mk, mv, mdk, mdv, a, ds, part);
  else
    window_dkv_kernel<D, F16, false><<<grid, kWbThreads, smem, st>>>(mq, mg, mk, mv, mdk, mdv, a, ds, part);
  if (cudaGetLastError() != cudaSuccess) return VSA_ERR_CUDA;
  if (ds.tiles() > 0) {
    const int shared = ds.sn > 1 ? ds.blocks : ds.heavy;
    window_dkv_sum_kernel<D, F16><<<dim3(shared * (D / 4), a.Hkv, a.B), 256, 0, st>>>(a, ds, part);
  }
  return cudaGetLastError() == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
}

}  // namespace vsa

using namespace vsa;

extern "C" {

size_t vsa_window_attn_workspace_bytes(const vsa_window* w) {
  WinArgs a;
  if (win_args(w, 1.f, &a) != VSA_OK) return 0;
  return win_fwd_bytes(a, w->d, win_plan(a).partial());
}

int vsa_window_attn(const vsa_window* w, const void* q, const void* k, const void* v, float softmax_scale, void* o,
                    float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  WinArgs a;
  int rc = win_args(w, softmax_scale, &a);
  if (rc != VSA_OK) return rc;
  if (q == nullptr || k == nullptr || v == nullptr || o == nullptr || lse == nullptr) return VSA_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(o, 16) || !aligned_to(lse, 4) ||
      !aligned_to(workspace, 16))
    return VSA_ERR_ALIGNMENT;
  const WinPlan plan = win_plan(a);
  const size_t need = win_fwd_bytes(a, w->d, plan.partial());
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return VSA_ERR_WORKSPACE;
  if ((rc = check_arch()) != VSA_OK) return rc;
  if ((a.err = device_error_ptr()) == nullptr) return VSA_ERR_CUDA;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.out = static_cast<uint16_t*>(o);
  a.lse = lse;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f16 = w->dtype == VSA_DTYPE_F16;
  float* part = static_cast<float*>(workspace);
  if (w->d == 128) return f16 ? launch_any<128, true>(a, plan, part, st) : launch_any<128, false>(a, plan, part, st);
  return f16 ? launch_any<64, true>(a, plan, part, st) : launch_any<64, false>(a, plan, part, st);
}

size_t vsa_window_attn_bwd_workspace_bytes(const vsa_window* w) {
  WinArgs a;
  if (win_args(w, 1.f, &a) != VSA_OK || win_bwd_strides(w, &a) != VSA_OK) return 0;
  return win_bwd_bytes(w, dkv_split(a));
}

int vsa_window_attn_bwd(const vsa_window* w, const void* d_o, const void* q, const void* k, const void* v,
                        const void* o, const float* lse, float softmax_scale, void* dq, void* dk, void* dv,
                        void* workspace, size_t workspace_bytes, void* stream) {
  WinArgs a;
  int rc = win_args(w, softmax_scale, &a);
  if (rc != VSA_OK || (rc = win_bwd_strides(w, &a)) != VSA_OK) return rc;
  const void* ptrs[] = {d_o, q, k, v, o, dq, dk, dv};
  for (const void* p : ptrs)
    if (p == nullptr) return VSA_ERR_INVALID_ARG;
  if (lse == nullptr) return VSA_ERR_INVALID_ARG;
  for (const void* p : ptrs)
    if (!aligned_to(p, 16)) return VSA_ERR_ALIGNMENT;
  if (!aligned_to(lse, 4) || !aligned_to(workspace, 16)) return VSA_ERR_ALIGNMENT;
  const DkvSplit ds = dkv_split(a);
  if (workspace == nullptr || workspace_bytes < win_bwd_bytes(w, ds)) return VSA_ERR_WORKSPACE;
  if ((rc = check_arch()) != VSA_OK) return rc;
  if ((a.err = device_error_ptr()) == nullptr) return VSA_ERR_CUDA;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.o = static_cast<const uint16_t*>(o);
  a.d_o = static_cast<const uint16_t*>(d_o);
  a.lse = const_cast<float*>(lse);
  a.dq = static_cast<uint16_t*>(dq);
  a.dk = static_cast<uint16_t*>(dk);
  a.dv = static_cast<uint16_t*>(dv);
  a.delta = static_cast<float*>(workspace);
  unsigned char* ws = static_cast<unsigned char*>(workspace) + win_delta_bytes(w);
  a.grad_bound = reinterpret_cast<unsigned int*>(ws);
  a.v_norms = reinterpret_cast<float*>(ws) + static_cast<size_t>(w->B) * w->Hkv;
  a.chunks = win_chunks(w);
  float* part = reinterpret_cast<float*>(ws + win_range_bytes(w));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f16 = w->dtype == VSA_DTYPE_F16;
  if (w->d == 128) return f16 ? launch_bwd<128, true>(a, ds, part, st) : launch_bwd<128, false>(a, ds, part, st);
  return f16 ? launch_bwd<64, true>(a, ds, part, st) : launch_bwd<64, false>(a, ds, part, st);
}

}  // extern "C"

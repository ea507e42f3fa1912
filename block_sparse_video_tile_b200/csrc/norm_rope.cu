// norm_rope.cu -- vsa_qk_norm_rope and its gradient: argument checks and
// launches (declared in include/vsa.h, kernels in norm_rope.cuh).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "norm_rope.cuh"
#include "vsa.h"
#include "vsa_host.h"

namespace vsa {

int take_strides(const int64_t in[3], int B, int N, int H, int d, long long out[3]) {
  const int extent[3] = {B, N, H};
  for (int i = 0; i < 3; ++i) {
    if (extent[i] == 1) {
      out[i] = d;
      continue;
    }
    if (in[i] <= 0) return VSA_ERR_INVALID_ARG;
    if (in[i] % 8 != 0) return VSA_ERR_ALIGNMENT;
    if (in[i] >= (1ll << 38)) return VSA_ERR_TOO_LARGE;
    out[i] = in[i];
  }
  return VSA_OK;
}

// CTAs of a launch, both sides together: two an SM (each backward CTA leaves
// one partial sum of dweight).
constexpr int kNrCtas = 148 * 2;
// A CTA walks all heads of its tokens if that gives this many items a side;
// below it the heads are split into chunks of kNrChunk or more.
constexpr int kNrWantItems = 148 * 8;

static int nr_side(const vsa_norm_rope* p, const vsa_qk_side* in, bool bwd, NrSide* s) {
  if (in->B <= 0 || in->H <= 0 || in->T <= 0 || in->Hh <= 0 || in->W <= 0) return VSA_ERR_INVALID_ARG;
  if (in->x == nullptr || in->y == nullptr) return VSA_ERR_INVALID_ARG;
  if (bwd && (in->dx == nullptr || (in->weight == nullptr) != (in->dweight == nullptr))) return VSA_ERR_INVALID_ARG;
  const long long N = 1ll * in->T * in->Hh;
  if (N > (1ll << 30) || N * in->W > (1ll << 30)) return VSA_ERR_TOO_LARGE;
  s->N = static_cast<int>(N * in->W);
  s->H = in->H;
  s->Hh = in->Hh;
  s->W = in->W;
  int rc;
  if ((rc = take_strides(in->x_s, in->B, s->N, in->H, p->d, s->xs)) != VSA_OK ||
      (rc = take_strides(in->y_s, in->B, s->N, in->H, p->d, bwd ? s->ys : s->os)) != VSA_OK)
    return rc;
  if (bwd && (rc = take_strides(in->dx_s, in->B, s->N, in->H, p->d, s->os)) != VSA_OK) return rc;
  if (!aligned_to(in->x, 16) || !aligned_to(in->y, 16) || !aligned_to(in->weight, 16) || !aligned_to(in->table, 8) ||
      (bwd && (!aligned_to(in->dx, 16) || !aligned_to(in->dweight, 4))))
    return VSA_ERR_ALIGNMENT;
  s->x = static_cast<const uint16_t*>(in->x);
  s->dy = bwd ? static_cast<const uint16_t*>(in->y) : nullptr;
  s->out = static_cast<uint16_t*>(bwd ? in->dx : in->y);
  s->weight = in->weight;
  s->weight_f32 = in->weight_f32;
  s->table = reinterpret_cast<const float2*>(in->table);
  const long long rows = 1ll * in->T * (p->split[0] / 2) + 1ll * in->Hh * (p->split[1] / 2);
  if (rows > 0x7fffffffll) return VSA_ERR_TOO_LARGE;
  s->toff1 = static_cast<int>(1ll * in->T * (p->split[0] / 2));
  s->toff2 = static_cast<int>(rows);
  s->partial = nullptr;
  const int lane_groups = 512 / p->d;                  // of a warp
  s->across = s->xs[2] < s->xs[1] && in->H >= kNrRows * lane_groups;
  const int tok = kNrThreads / 32 * (s->across ? 1 : lane_groups);
  s->groups = (s->N + tok - 1) / tok;
  const long long whole = 1ll * in->B * s->groups;
  s->chunks = 1;
  const int least = s->across ? kNrRows * lane_groups : kNrChunk;
  if (whole < kNrWantItems) {
    const long long most = (in->H + least - 1) / least;
    s->chunks = static_cast<int>(std::min<long long>(most, (kNrWantItems + whole - 1) / whole));
  }
  s->hpc = ((in->H + s->chunks - 1) / s->chunks + least - 1) / least * least;
  s->chunks = (in->H + s->hpc - 1) / s->hpc;
  if (whole * s->chunks > (1ll << 30)) return VSA_ERR_TOO_LARGE;   // the kernel's item index steps by the grid in 32 bits
  s->items = static_cast<int>(whole * s->chunks);
  return VSA_OK;
}

static int nr_args(const vsa_norm_rope* p, const vsa_qk_side* q, const vsa_qk_side* k, bool bwd, NrArgs* a) {
  if (p == nullptr || q == nullptr) return VSA_ERR_INVALID_ARG;
  if (p->d != 64 && p->d != 128) return VSA_ERR_UNSUPPORTED;
  if (p->dtype != VSA_DTYPE_BF16 && p->dtype != VSA_DTYPE_F16) return VSA_ERR_UNSUPPORTED;
  if (!(p->eps >= 0.f) || !std::isfinite(p->eps)) return VSA_ERR_INVALID_ARG;
  long long sum = 0;
  for (int i = 0; i < 3; ++i) {
    if (p->split[i] < 0 || p->split[i] % 2 != 0) return VSA_ERR_INVALID_ARG;
    sum += p->split[i];
  }
  if (sum != p->d) return VSA_ERR_INVALID_ARG;
  a->c0 = p->split[0] / 2;
  a->c1 = p->split[1] / 2;
  a->c2 = p->split[2] / 2;
  a->eps = p->eps;
  int rc = nr_side(p, q, bwd, &a->s[0]);
  if (rc != VSA_OK) return rc;
  a->s[1] = a->s[0];
  a->s[1].items = 0;
  return k != nullptr ? nr_side(p, k, bwd, &a->s[1]) : VSA_OK;
}

// CTAs a side (grid.x).
static int nr_ctas(const NrArgs& a) {
  return std::min(a.s[1].items > 0 ? kNrCtas / 2 : kNrCtas, std::max(a.s[0].items, a.s[1].items));
}

template <bool BWD>
static int nr_launch(const vsa_norm_rope* p, const NrArgs& a, int ctas, int sides, cudaStream_t st) {
  const dim3 grid(ctas, sides);
  const bool f16 = p->dtype == VSA_DTYPE_F16, il = p->interleaved != 0;
  constexpr int smem = nr_smem_bytes<BWD>();
#define VSA_NR(D, F, I)                                                                                        \
  do {                                                                                                         \
    if (cudaFuncSetAttribute(norm_rope_kernel<D, F, I, BWD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != \
        cudaSuccess)                                                                                           \
      return VSA_ERR_CUDA;                                                                                     \
    norm_rope_kernel<D, F, I, BWD><<<grid, kNrThreads, smem, st>>>(a);                                         \
  } while (0)
  if (p->d == 128) {
    if (f16) { if (il) VSA_NR(128, true, true); else VSA_NR(128, true, false); }
    else { if (il) VSA_NR(128, false, true); else VSA_NR(128, false, false); }
  } else {
    if (f16) { if (il) VSA_NR(64, true, true); else VSA_NR(64, true, false); }
    else { if (il) VSA_NR(64, false, true); else VSA_NR(64, false, false); }
  }
#undef VSA_NR
  return cudaGetLastError() == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
}


static size_t nr_bwd_bytes(const vsa_norm_rope* p, const NrArgs& a, const vsa_qk_side* q, const vsa_qk_side* k) {
  const size_t sides = (q->weight != nullptr ? 1 : 0) + (k != nullptr && k->weight != nullptr ? 1 : 0);
  return sides * nr_ctas(a) * p->d * sizeof(float);
}

}  // namespace vsa

using namespace vsa;

extern "C" {

int vsa_qk_norm_rope(const vsa_norm_rope* p, const vsa_qk_side* q, const vsa_qk_side* k, void* stream) {
  NrArgs a;
  int rc = nr_args(p, q, k, false, &a);
  if (rc != VSA_OK) return rc;
  if ((rc = check_arch()) != VSA_OK) return rc;
  return nr_launch<false>(p, a, nr_ctas(a), k != nullptr ? 2 : 1, static_cast<cudaStream_t>(stream));
}

size_t vsa_qk_norm_rope_bwd_workspace_bytes(const vsa_norm_rope* p, const vsa_qk_side* q, const vsa_qk_side* k) {
  NrArgs a;
  return nr_args(p, q, k, true, &a) == VSA_OK ? nr_bwd_bytes(p, a, q, k) : 0;
}

int vsa_qk_norm_rope_bwd(const vsa_norm_rope* p, const vsa_qk_side* q, const vsa_qk_side* k, void* workspace,
                         size_t workspace_bytes, void* stream) {
  NrArgs a;
  int rc = nr_args(p, q, k, true, &a);
  if (rc != VSA_OK) return rc;
  const size_t need = nr_bwd_bytes(p, a, q, k);
  if (!aligned_to(workspace, 16)) return VSA_ERR_ALIGNMENT;
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return VSA_ERR_WORKSPACE;
  if ((rc = check_arch()) != VSA_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int ctas = nr_ctas(a);
  float* ws = static_cast<float*>(workspace);
  if (q->weight != nullptr) {
    a.s[0].partial = ws;
    ws += static_cast<size_t>(ctas) * p->d;
  }
  const bool kw = k != nullptr && k->weight != nullptr;
  if (kw) a.s[1].partial = ws;
  if ((rc = nr_launch<true>(p, a, ctas, k != nullptr ? 2 : 1, st)) != VSA_OK || need == 0) return rc;
  float* dk = kw ? k->dweight : nullptr;
  if (p->d == 128)
    norm_rope_dweight_kernel<128><<<2, 1024, 0, st>>>(a.s[0].partial, q->dweight, a.s[1].partial, dk, ctas);
  else
    norm_rope_dweight_kernel<64><<<2, 1024, 0, st>>>(a.s[0].partial, q->dweight, a.s[1].partial, dk, ctas);
  return cudaGetLastError() == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
}

}  // extern "C"

// fp8_block_api.cu -- the entry points of the block-scaled FP8 operators:
// argument checks, the choice of kernel, the launches.  Declarations and
// argument contracts: include/dfk.h.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "api_internal.h"
#include "dfk.h"
#include "fp8_block.cuh"
#include "launch_util.h"

namespace dfk {

static bool off16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
static bool off4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

static int check_rows(int M, int K) {
  if (M < 0 || K <= 0) return api_fail(DFK_ERR_INVALID_ARG, "negative or zero size");
  if (K % 16) return api_fail(DFK_ERR_UNSUPPORTED_SHAPE, "row length %% 16 != 0 (%d)", K);
  return DFK_OK;
}

constexpr int FB_SMEM_MAX = 232448;     // bytes a CTA may use
constexpr int FB_SMEM_HALF = 115712;    // two CTAs on an SM

// Up to this many tokens a product streams its weights (fp8_block_small.cu).
constexpr int FB_SMALL_MAX_M = 64;

struct FbCall {
  int nmat;
  const void *qx;
  const float *sx;
  const void *qw[2];
  const float *sw[2];
  void *y, *qh;
  float *sh;
  int M, K, N;
};

static int launch_small(const FbCall &c, int sms, unsigned *err, cudaStream_t st) {
  const int G = (c.K + FB_GROUP - 1) / FB_GROUP;
  const int bn = c.M <= 16 ? 16 : c.M <= 32 ? 32 : 64;
  const int blocks = (c.N + 127) / 128, tiles = (c.M + bn - 1) / bn;
  if (tiles > 65535) return api_fail(DFK_ERR_UNSUPPORTED_SHAPE, "M=%d is too large", c.M);
  // Clusters of 1, 2, 4 or 8 CTAs a row block, each with four groups or more.
  // One matrix: up to two CTAs on an SM, so that the next call's weights load
  // while this one ends (N = 6144, K = 4096: 7.3 us against 9.1 at one CTA;
  // clusters of 3, as many as fill the SMs, 15.5: they do not all fit at once).
  // Two matrices: one CTA on an SM with all of its shared memory (stages of
  // 32 KB and more), two where the row blocks outnumber the SMs.
  const long long work = static_cast<long long>(blocks) * tiles;
  const bool pack = c.nmat == 1 || (bn < 64 && work > sms);
  const int limit = pack ? 2 * sms : sms;
  int ks = 1;
  while (ks < 8 && work * ks * 2 <= limit && ks * 8 <= G) ks *= 2;
  const int cap = pack ? FB_SMEM_HALF : FB_SMEM_MAX;
  int stages = fb_small_min_stages(c.nmat, bn);
  const int most = (G + ks - 1) / ks;
  while (stages < 16 && stages < most && fb_small_smem(c.nmat, bn, stages + 1) <= cap) ++stages;
  const void *fn = fb_small_kernel(c.nmat, bn);
  int rc = api_allow_smem(fn);
  if (rc) return rc;
  FbMaps maps;
  memset(&maps, 0, sizeof maps);
  if ((rc = api_tensor_map_u8(c.qx, c.K, c.M, c.K, 128, bn, &maps.x))) return rc;
  for (int m = 0; m < c.nmat; ++m)
    if ((rc = api_tensor_map_u8(c.qw[m], c.K, c.N, c.K, 128, 128, &maps.w[m]))) return rc;
  FbParams p{c.sx, {c.sw[0], c.sw[1]}, static_cast<uint16_t *>(c.y),
             static_cast<uint8_t *>(c.qh), c.sh, err, c.M, c.N, G, stages};
  void *args[] = {&maps, &p};
  const cudaError_t e = launch_kernel(
      fn, dim3(static_cast<unsigned>(blocks * ks), tiles), dim3(fb_small_threads(c.nmat, bn)),
      fb_small_smem(c.nmat, bn, stages), st, api_pdl(), args, static_cast<unsigned>(ks));
  if (e != cudaSuccess) return api_cuda_error(e, "block-scaled FP8 product launch");
  return DFK_OK;
}

static int launch_large(const FbCall &c, int sms, unsigned *err, cudaStream_t st) {
  const bool gate = c.nmat == 2;
  const int G = (c.K + FB_GROUP - 1) / FB_GROUP;
  const long long tn = gate ? (c.N + 127) / 128 : (c.N + 255) / 256;
  const long long singles = (c.M + 127LL) / 128 * tn, pairs = (c.M + 255LL) / 256 * tn;
  // The form with fewer rounds of tiles over the SMs; pairs, which read a
  // third less per product, where both need as many.
  const bool pair = (singles + sms - 1) / sms >= (pairs + sms / 2 - 1) / (sms / 2) && pairs > sms / 4;
  int ks = 1;
  if (!pair)
    while (ks < 8 && singles * ks * 2 <= sms && ks * 8 <= G) ks *= 2;
  int rc = api_allow_smem(fb_large_kernel_fn(gate, pair));
  if (rc) return rc;
  FbMaps maps;
  memset(&maps, 0, sizeof maps);
  if ((rc = api_tensor_map_u8(c.qx, c.K, c.M, c.K, 128, 128, &maps.x))) return rc;
  for (int m = 0; m < c.nmat; ++m)
    if ((rc = api_tensor_map_u8(c.qw[m], c.K, c.N, c.K, 128, fb_large_weight_box(pair),
                                &maps.w[m])))
      return rc;
  const FbParams p{c.sx, {c.sw[0], c.sw[1]}, static_cast<uint16_t *>(c.y),
                   static_cast<uint8_t *>(c.qh), c.sh, err, c.M, c.N, G, 0};
  const cudaError_t e = launch_fb_large(gate, pair, ks, maps, p, sms, st, api_pdl());
  if (e != cudaSuccess) return api_cuda_error(e, "block-scaled FP8 product launch");
  return DFK_OK;
}

static int product(const FbCall &c, cudaStream_t st) {
  int rc = check_rows(c.M, c.K);
  if (rc) return rc;
  if (c.N <= 0) return api_fail(DFK_ERR_INVALID_ARG, "negative or zero size");
  if (c.qh || c.sh) {
    if (c.y) return api_fail(DFK_ERR_INVALID_ARG, "both a bf16 and a quantised output");
    if (c.N % 16)
      return api_fail(DFK_ERR_UNSUPPORTED_SHAPE, "quantised output: row length %% 16 != 0 (%d)",
                      c.N);
  }
  if (c.M == 0) return DFK_OK;
  if (!c.qx || !c.sx || !(c.y || (c.qh && c.sh)))
    return api_fail(DFK_ERR_INVALID_ARG, "null pointer argument");
  if (off16(c.qx) || off16(c.y) || off16(c.qh))
    return api_fail(DFK_ERR_MISALIGNED, "device pointers must be 16-byte aligned");
  if (off4(c.sx) || off4(c.sh))
    return api_fail(DFK_ERR_MISALIGNED, "scale pointers must be 4-byte aligned");
  for (int m = 0; m < c.nmat; ++m) {
    if (!c.qw[m] || !c.sw[m]) return api_fail(DFK_ERR_INVALID_ARG, "null pointer argument");
    if (off16(c.qw[m]))
      return api_fail(DFK_ERR_MISALIGNED, "device pointers must be 16-byte aligned");
    if (off4(c.sw[m]))
      return api_fail(DFK_ERR_MISALIGNED, "scale pointers must be 4-byte aligned");
  }
  int sms;
  unsigned *err;
  if ((rc = api_device(&sms, &err))) return rc;
  return c.M <= FB_SMALL_MAX_M ? launch_small(c, sms, err, st) : launch_large(c, sms, err, st);
}

}  // namespace dfk

using namespace dfk;

extern "C" {

int dfk_quant_fp8_block(const void *x, void *q, float *s, int M, int K, void *stream) {
  int rc = check_rows(M, K);
  if (rc || M == 0) return rc;
  if (!x || !q || !s) return api_fail(DFK_ERR_INVALID_ARG, "null pointer argument");
  if (off16(x) || off16(q))
    return api_fail(DFK_ERR_MISALIGNED, "device pointers must be 16-byte aligned");
  if (off4(s)) return api_fail(DFK_ERR_MISALIGNED, "scale pointers must be 4-byte aligned");
  int sms;
  unsigned *err;
  if ((rc = api_device(&sms, &err))) return rc;
  const cudaError_t e =
      launch_fb_quant(x, q, s, M, K, err, static_cast<cudaStream_t>(stream), api_pdl());
  return e == cudaSuccess ? DFK_OK : api_cuda_error(e, "block quantisation launch");
}

int dfk_add_rmsnorm_fp8_block(const void *x, const void *residual, const void *gamma, float eps,
                              void *residual_out, void *q, float *s, int M, int d_model,
                              void *stream) {
  int rc = check_rows(M, d_model);
  if (rc) return rc;
  if (!(eps >= 0.f && std::isfinite(eps)))
    return api_fail(DFK_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (d_model > FB_NORM_MAX_D)
    return api_fail(DFK_ERR_UNSUPPORTED_SHAPE, "d_model=%d > %d", d_model, FB_NORM_MAX_D);
  if (M == 0) return DFK_OK;
  if (!x || !gamma || !q || !s || (residual && !residual_out))
    return api_fail(DFK_ERR_INVALID_ARG, "null pointer argument");
  if (!residual && residual_out)
    return api_fail(DFK_ERR_INVALID_ARG, "residual_out without a residual");
  if (off16(x) || off16(residual) || off16(gamma) || off16(residual_out) || off16(q))
    return api_fail(DFK_ERR_MISALIGNED, "device pointers must be 16-byte aligned");
  if (off4(s)) return api_fail(DFK_ERR_MISALIGNED, "scale pointers must be 4-byte aligned");
  int sms;
  unsigned *err;
  if ((rc = api_device(&sms, &err))) return rc;
  const cudaError_t e = launch_fb_norm(x, residual, gamma, eps, residual_out, q, s, M, d_model,
                                       err, static_cast<cudaStream_t>(stream), api_pdl());
  return e == cudaSuccess ? DFK_OK : api_cuda_error(e, "RMSNorm quantisation launch");
}

int dfk_gemm_fp8_block(const void *q_x, const float *s_x, const void *q_w, const float *s_w,
                       void *y, int M, int K, int N, void *stream) {
  const FbCall c{1, q_x, s_x, {q_w, nullptr}, {s_w, nullptr}, y, nullptr, nullptr, M, K, N};
  return product(c, static_cast<cudaStream_t>(stream));
}

int dfk_swiglu_gate_up_fp8_block(const void *q_x, const float *s_x, const void *q_gate,
                                 const float *s_gate, const void *q_up, const float *s_up,
                                 void *h, void *q_h, float *s_h, int M, int d_model, int d_ff,
                                 void *stream) {
  const FbCall c{2, q_x, s_x, {q_gate, q_up}, {s_gate, s_up}, h, q_h, s_h, M, d_model, d_ff};
  return product(c, static_cast<cudaStream_t>(stream));
}

}  // extern "C"

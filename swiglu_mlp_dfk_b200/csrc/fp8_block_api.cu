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

// Sizes the kernels' 32-bit coordinates hold with a tile to spare.
constexpr int FB_MAX_SIZE = 0x7fffffff - 1023;

static int check_rows(int M, int K) {
  if (M < 0 || K <= 0) return api_fail(DFK_ERR_INVALID_ARG, "negative or zero size");
  if (M > FB_MAX_SIZE || K > FB_MAX_SIZE)
    return api_fail(DFK_ERR_UNSUPPORTED_SHAPE, "%d x %d: a size is too large", M, K);
  if (K % 16) return api_fail(DFK_ERR_UNSUPPORTED_SHAPE, "row length %% 16 != 0 (%d)", K);
  return DFK_OK;
}

constexpr int FB_SMEM_MAX = 232448;     // bytes a CTA may use
constexpr int FB_SMEM_HALF = 115712;    // two CTAs on an SM

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

// ---- which kernel, in which form

static int ceil_div(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

// The streaming kernel (fp8_block_small.cu): tokens of a tile, CTAs of a row block,
// two CTAs on an SM or one.  Clusters of 1, 2, 4 or 8 CTAs a row block, each with
// four groups or more.  One matrix: two CTAs on an SM, so that the next call's
// weights load while this one ends (16 tokens, N = 6144, K = 4096: 7.3 us against
// 9.1 at one CTA; clusters of 3, as many as fill the SMs, 15.5: they do not all
// fit at once).  Two matrices: one CTA on an SM with all of its shared memory
// (stages of 32 KB and more), two where the row blocks outnumber the SMs.
// Clusters of 8 that have their SMs to themselves find room on three quarters of
// them, no more (K = 4096, 1 token: d_ff = 1920 7.4 us, 2048 12.1, 7.2 in clusters of 4), and
// above 16 tokens their meeting costs more than four groups less (24 tokens, d_ff =
// 1024: K = 4096 8.5 us, 7.8 in clusters of 4; K = 8192 10.4 and 11.0).
struct SmallPlan {
  int bn, blocks, tiles, ks, stages;
  bool pack;
  double us;
};

static SmallPlan plan_small(const FbCall &c, int G, int sms) {
  SmallPlan s;
  s.bn = c.M <= 16 ? 16 : c.M <= 32 ? 32 : 64;
  s.blocks = ceil_div(c.N, 128);
  s.tiles = ceil_div(c.M, s.bn);
  const long long work = static_cast<long long>(s.blocks) * s.tiles;
  s.pack = c.nmat == 1 || (s.bn < 64 && work > sms);
  const int limit = s.pack ? 2 * sms : sms;
  s.ks = 1;
  while (s.ks < 8 && work * s.ks * 2 <= limit && s.ks * 8 <= G) s.ks *= 2;
  if (!s.pack && s.ks == 8 && (work * 8 > sms * 3 / 4 || (s.bn > 16 && G < 64))) s.ks = 4;
  const int waves = ceil_div(work * s.ks, limit);
  s.us = 1.9 + (2.6 + 0.53 * ceil_div(G, s.ks)) * waves;
  const int cap = s.pack ? FB_SMEM_HALF : FB_SMEM_MAX, most = ceil_div(G, s.ks);
  s.stages = fb_small_min_stages(c.nmat, s.bn);
  while (s.stages < 16 && s.stages < most &&
         fb_small_smem(c.nmat, s.bn, s.stages + 1) <= cap)
    ++s.stages;
  return s;
}

// The tensor-bound kernel (fp8_block_large.cu): tiles of 256 tokens by pairs of
// CTAs, or of 128 tokens by single CTAs or clusters of ks of them.  Clusters of
// 8 do not all fit on the SMs (96 tokens, N = 4096, K = 14336: 34 us, 22 with 4).
struct LargePlan {
  bool pair;
  int ks;
  double us;
};

static LargePlan plan_large(const FbCall &c, int G, int sms) {
  const long long tn = ceil_div(c.N, c.nmat == 2 ? 128 : 256);
  const long long singles = ceil_div(c.M, 128) * tn, pairs = ceil_div(c.M, 256) * tn;
  LargePlan best{true, 1, 4.0 + (2.0 + 0.36 * G) * ceil_div(pairs, sms / 2)};
  for (int ks = 1; ks <= 4 && ks * 4 <= std::max(G, 4); ks *= 2) {
    if (ks > 1 && singles * ks > sms * 9 / 10) break;
    const double us =
        (ks > 1 ? 8.0 : 4.0) + (2.0 + 0.42 * ceil_div(G, ks)) * ceil_div(singles * ks, sms);
    if (us < best.us) best = LargePlan{false, ks, us};
  }
  return best;
}

// `us` above ranks the forms of one product and tells no more than that (gate/up of
// 4096 tokens, K = 4096, d_ff = 14336: 342 here, 424 measured in a burst).  It was
// fitted to calls of 48 to 8192 tokens on a B200: a fixed part (launch, first loads;
// 4 us more where a cluster adds its shares), a part per round of tiles (their
// output, which the next tile's groups do not hide) and a part per group of a round.
// Both sides measured at 192 tokens: N = 6144, K = 4096 14.0 us streaming, 17.8 by
// pairs; N = 4096, K = 14336 33.6 us streaming, 23.1 by clusters of 4, 46.5 by pairs;
// N = 16384, K = 4096 41, 21.5, 20.  8192 tokens, N = 1024, K = 128: 13.6 streaming,
// 9.4 by pairs, 9.7 by single CTAs.
struct Plan {
  SmallPlan small;
  LargePlan large;
  bool streams;  // the streaming kernel
};

// Up to 64 tokens the weights' bytes bound every form: the streaming kernel.
static Plan choose(const FbCall &c, int G, int sms) {
  Plan p{plan_small(c, G, sms), plan_large(c, G, sms), true};
  p.streams = c.M <= 64 || p.small.us <= p.large.us;
  return p;
}

static int launch_small(const FbCall &c, const SmallPlan &s, int G, unsigned *err,
                        cudaStream_t st) {
  if (s.tiles > 65535) return api_fail(DFK_ERR_UNSUPPORTED_SHAPE, "M=%d is too large", c.M);
  const void *fn = fb_small_kernel(c.nmat, s.bn);
  int rc = api_allow_smem(fn);
  if (rc) return rc;
  FbMaps maps;
  memset(&maps, 0, sizeof maps);
  if ((rc = api_tensor_map_u8(c.qx, c.K, c.M, c.K, 128, s.bn, &maps.x))) return rc;
  for (int m = 0; m < c.nmat; ++m)
    if ((rc = api_tensor_map_u8(c.qw[m], c.K, c.N, c.K, 128, 128, &maps.w[m]))) return rc;
  FbParams p{c.sx, {c.sw[0], c.sw[1]}, static_cast<uint16_t *>(c.y),
             static_cast<uint8_t *>(c.qh), c.sh, err, c.M, c.N, G, s.stages, 0};
  void *args[] = {&maps, &p};
  const cudaError_t e = launch_kernel(
      fn, dim3(static_cast<unsigned>(s.blocks) * s.ks, s.tiles),
      dim3(fb_small_threads(c.nmat, s.bn)), fb_small_smem(c.nmat, s.bn, s.stages), st, api_pdl(),
      args, static_cast<unsigned>(s.ks));
  if (e != cudaSuccess) return api_cuda_error(e, "block-scaled FP8 product launch");
  return DFK_OK;
}

static int launch_large(const FbCall &c, const LargePlan &l, int G, int sms, unsigned *err,
                        cudaStream_t st) {
  const bool gate = c.nmat == 2;
  int rc = api_allow_smem(fb_large_kernel_fn(gate, l.pair));
  if (rc) return rc;
  FbMaps maps;
  memset(&maps, 0, sizeof maps);
  if ((rc = api_tensor_map_u8(c.qx, c.K, c.M, c.K, 128, 128, &maps.x))) return rc;
  for (int m = 0; m < c.nmat; ++m)
    if ((rc = api_tensor_map_u8(c.qw[m], c.K, c.N, c.K, 128, fb_large_weight_box(l.pair),
                                &maps.w[m])))
      return rc;
  const FbParams p{c.sx, {c.sw[0], c.sw[1]}, static_cast<uint16_t *>(c.y),
                   static_cast<uint8_t *>(c.qh), c.sh, err, c.M, c.N, G, 0, 0};
  const cudaError_t e = launch_fb_large(gate, l.pair, l.ks, maps, p, sms, st, api_pdl());
  if (e != cudaSuccess) return api_cuda_error(e, "block-scaled FP8 product launch");
  return DFK_OK;
}

static int product(const FbCall &c, cudaStream_t st) {
  int rc = check_rows(c.M, c.K);
  if (rc) return rc;
  if (c.N <= 0) return api_fail(DFK_ERR_INVALID_ARG, "negative or zero size");
  if (c.N > FB_MAX_SIZE)
    return api_fail(DFK_ERR_UNSUPPORTED_SHAPE, "%d weight rows: too large", c.N);
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
  const int G = ceil_div(c.K, FB_GROUP);
  const Plan plan = choose(c, G, sms);
  return plan.streams ? launch_small(c, plan.small, G, err, st)
                      : launch_large(c, plan.large, G, sms, err, st);
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

// For the tests, which name the forms that they run; not part of dfk.h.  The form of
// a product with nmat weight matrices on `sms` SMs: {1, tokens of a tile, CTAs of a
// row block, two CTAs an SM, ring stages} of the streaming kernel, or {0, pairs of
// CTAs, CTAs of a tile, 0, 0} of the tensor-bound one.
__attribute__((visibility("default"))) void dfk_fp8_block_form(int nmat, int M, int K, int N,
                                                               int sms, int form[5]) {
  FbCall c{};
  c.nmat = nmat;
  c.M = M;
  c.K = K;
  c.N = N;
  const Plan p = choose(c, ceil_div(K, FB_GROUP), sms);
  const int streams[5] = {1, p.small.bn, p.small.ks, p.small.pack, p.small.stages};
  const int bound[5] = {0, p.large.pair, p.large.pair ? 2 : p.large.ks, 0, 0};
  memcpy(form, p.streams ? streams : bound, sizeof streams);
}

}  // extern "C"

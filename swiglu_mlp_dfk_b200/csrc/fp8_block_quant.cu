// fp8_block_quant.cu -- activations into block-scaled FP8 (fp8_block.cuh):
// straight from bf16, and out of the RMSNorm with the residual's addition.
#include <algorithm>

#include "fp8_block.cuh"
#include "launch_util.h"

namespace dfk {

// max |v| over the 16 lanes that hold one group of 128 (8 elements a lane).
__device__ __forceinline__ float group_max(float a) {
#pragma unroll
  for (int m = 8; m >= 1; m >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, m));
  return a;
}

__device__ __forceinline__ float abs_max8(const float (&v)[8]) {
  float a = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) a = max_nan(a, fabsf(v[i]));
  return a;
}

__device__ __forceinline__ void unpack8(const uint4 &w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(u[i]);
    v[2 * i + 1] = bf16_hi(u[i]);
  }
}

constexpr int FBQ_THREADS = 256;
constexpr int FBQ_ROWS = 4;

// Half a warp takes one group of 128 of FBQ_ROWS consecutive rows: 16 bytes a
// lane and row, every load issued before the first use.
__global__ void __launch_bounds__(FBQ_THREADS)
    fb_quant_kernel(const uint16_t *__restrict__ x, uint8_t *__restrict__ q,
                    float *__restrict__ s, int M, int K, int G, long long items, unsigned *err) {
  const long long item =
      (static_cast<long long>(blockIdx.x) * FBQ_THREADS + threadIdx.x) >> 4;
  const int l = threadIdx.x & 15;
  pdl_launch_dependents();
  pdl_wait();
  const bool live = item < items;  // the shuffles below take every lane
  const int m0 = live ? static_cast<int>(item / G) * FBQ_ROWS : M;
  const int g = live ? static_cast<int>(item % G) : 0;
  const int k = g * FB_GROUP + 8 * l;
  const bool in = k < K;  // K % 16 == 0: a lane's 8 elements are all inside or all outside
  uint4 w[FBQ_ROWS];
#pragma unroll
  for (int r = 0; r < FBQ_ROWS; ++r) {
    w[r] = make_uint4(0u, 0u, 0u, 0u);
    if (in && m0 + r < M && DFK_IN_BOUNDS(k + 8 <= K, 20, err))
      w[r] = ld_nc_v4(x + static_cast<size_t>(m0 + r) * K + k);
  }
#pragma unroll
  for (int r = 0; r < FBQ_ROWS; ++r) {
    float v[8];
    unpack8(w[r], v);
    const FbScale f = fb_scale(group_max(abs_max8(v)));
    if (m0 + r < M) {
      if (in && DFK_IN_BOUNDS(k + 8 <= K, 21, err))
        *reinterpret_cast<uint2 *>(q + static_cast<size_t>(m0 + r) * K + k) =
            make_uint2(fb_codes4(v[0], v[1], v[2], v[3], f), fb_codes4(v[4], v[5], v[6], v[7], f));
      if (l == 0 && DFK_IN_BOUNDS(g < G, 22, err))
        s[static_cast<size_t>(g) * M + m0 + r] = f.s;
    }
  }
}

// One CTA per row; thread t holds chunks t + T i (8 elements each, i < CPT)
// of the row in registers, so every input is read once:
//   r = bf16(x + residual)      (stored; the norm reads the rounded sum, as
//                                the next layer does)
//   v = (r / sqrt(mean r^2 + eps)) * gamma, fp32, quantised per group.
template <int CPT>
__global__ void __launch_bounds__(1024)
    fb_norm_kernel(const uint16_t *x, const uint16_t *res, const uint16_t *__restrict__ gamma,
                   float eps, uint16_t *res_out, uint8_t *__restrict__ q,
                   float *__restrict__ s, int M, int D, int G, unsigned *err) {
  __shared__ float s_part[32];
  const int tid = threadIdx.x, T = blockDim.x;
  const int m = blockIdx.x;
  uint4 g[CPT];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int k = 8 * (tid + T * i);
    g[i] = make_uint4(0u, 0u, 0u, 0u);
    if (k < D) g[i] = ld_nc_v4(gamma + k);
  }
  pdl_launch_dependents();
  pdl_wait();
  const size_t row = static_cast<size_t>(m) * D;
  uint4 a[CPT], b[CPT];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int k = 8 * (tid + T * i);
    a[i] = b[i] = make_uint4(0u, 0u, 0u, 0u);
    if (k < D && DFK_IN_BOUNDS(k + 8 <= D && m < M, 23, err)) {
      a[i] = *reinterpret_cast<const uint4 *>(x + row + k);
      if (res) b[i] = *reinterpret_cast<const uint4 *>(res + row + k);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int k = 8 * (tid + T * i);
    uint32_t *aw = &a[i].x, *bw = &b[i].x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (res) {
        const uint32_t lo = f32_to_bf16_bits(bf16_lo(aw[j]) + bf16_lo(bw[j]));
        const uint32_t hi = f32_to_bf16_bits(bf16_hi(aw[j]) + bf16_hi(bw[j]));
        aw[j] = lo | (hi << 16);
      }
      const float f0 = bf16_lo(aw[j]), f1 = bf16_hi(aw[j]);
      ss = fmaf(f0, f0, ss);
      ss = fmaf(f1, f1, ss);
    }
    if (res_out && k < D && DFK_IN_BOUNDS(k + 8 <= D && m < M, 24, err))
      *reinterpret_cast<uint4 *>(res_out + row + k) = a[i];
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
  if ((tid & 31) == 0) s_part[tid >> 5] = ss;
  __syncthreads();
  // every warp adds the warps' sums with the same butterfly: one barrier
  ss = (tid & 31) < (T >> 5) ? s_part[tid & 31] : 0.f;
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
  const float r = 1.0f / sqrtf(ss / static_cast<float>(D) + eps);
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int k = 8 * (tid + T * i);
    float v[8], w[8];
    unpack8(a[i], v);
    unpack8(g[i], w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = k < D ? (v[j] * r) * w[j] : 0.f;
    const FbScale f = fb_scale(group_max(abs_max8(v)));
    if (k < D) {
      if (DFK_IN_BOUNDS(k + 8 <= D && m < M, 25, err))
        *reinterpret_cast<uint2 *>(q + row + k) =
            make_uint2(fb_codes4(v[0], v[1], v[2], v[3], f), fb_codes4(v[4], v[5], v[6], v[7], f));
      if ((tid & 15) == 0 && DFK_IN_BOUNDS(k / FB_GROUP < G, 26, err))
        s[static_cast<size_t>(k / FB_GROUP) * M + m] = f.s;
    }
  }
}

cudaError_t launch_fb_quant(const void *x, void *q, float *s, int M, int K, unsigned *err,
                            cudaStream_t st, bool pdl) {
  const uint16_t *xp = static_cast<const uint16_t *>(x);
  uint8_t *qp = static_cast<uint8_t *>(q);
  int G = (K + FB_GROUP - 1) / FB_GROUP;
  long long items = static_cast<long long>((M + FBQ_ROWS - 1) / FBQ_ROWS) * G;
  const long long grid = (items * 16 + FBQ_THREADS - 1) / FBQ_THREADS;
  void *args[] = {&xp, &qp, &s, &M, &K, &G, &items, &err};
  return launch_kernel(reinterpret_cast<const void *>(&fb_quant_kernel),
                       dim3(static_cast<unsigned>(grid)), dim3(FBQ_THREADS), 0, st, pdl, args);
}

cudaError_t launch_fb_norm(const void *x, const void *res, const void *gamma, float eps,
                           void *res_out, void *q, float *s, int M, int D, unsigned *err,
                           cudaStream_t st, bool pdl) {
  const uint16_t *xp = static_cast<const uint16_t *>(x), *rp = static_cast<const uint16_t *>(res),
                 *gp = static_cast<const uint16_t *>(gamma);
  uint16_t *op = static_cast<uint16_t *>(res_out);
  uint8_t *qp = static_cast<uint8_t *>(q);
  int G = (D + FB_GROUP - 1) / FB_GROUP;
  const int chunks = D / 8;
  const int cpt = chunks <= 512 ? 1 : chunks <= 2048 ? 2 : 4;
  const int T = ((chunks + cpt - 1) / cpt + 31) / 32 * 32;
  const void *fn = cpt == 1   ? reinterpret_cast<const void *>(&fb_norm_kernel<1>)
                   : cpt == 2 ? reinterpret_cast<const void *>(&fb_norm_kernel<2>)
                              : reinterpret_cast<const void *>(&fb_norm_kernel<4>);
  void *args[] = {&xp, &rp, &gp, &eps, &op, &qp, &s, &M, &D, &G, &err};
  return launch_kernel(fn, dim3(M), dim3(T), 0, st, pdl, args);
}

}  // namespace dfk

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

__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// max |v| of eight bf16 values, in the low half.
__device__ __forceinline__ uint32_t bf16x2_abs_max(const uint4 &w) {
  const uint32_t m = 0x7fff7fffu;
  const uint32_t a = max_nan_bf16x2(max_nan_bf16x2(w.x & m, w.y & m),
                                    max_nan_bf16x2(w.z & m, w.w & m));
  return max_nan_bf16x2(a, a >> 16);
}

constexpr int FBQ_THREADS = 128;
constexpr int FBQ_ROWS = 4;

// Half a warp takes one group of 128 of FBQ_ROWS consecutive rows: 16 bytes a
// lane and row, every load issued before the first use.  Bound by memory: 2047
// rows of 14336 in 14.9 us, 91 % of the copy rate (17.2 us when every lane worked
// out every row's scale and maximum in fp32: 13 instructions an element).
__global__ void __launch_bounds__(FBQ_THREADS)
    fb_quant_kernel(const uint16_t *x, uint8_t *__restrict__ q,
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
      w[r] = fb_ld_v4(x + static_cast<size_t>(m0 + r) * K + k);
  }
  // Magnitudes stay in bf16 (exact) until the group's is known: two rows share
  // a register in the butterfly over the 16 lanes.
  uint32_t top[FBQ_ROWS / 2];
#pragma unroll
  for (int r = 0; r < FBQ_ROWS; r += 2)
    top[r / 2] = __byte_perm(bf16x2_abs_max(w[r]), bf16x2_abs_max(w[r + 1]), 0x5410);
#pragma unroll
  for (int d = 8; d >= 1; d >>= 1)
#pragma unroll
    for (int r = 0; r < FBQ_ROWS / 2; ++r)
      top[r] = max_nan_bf16x2(top[r], __shfl_xor_sync(0xffffffffu, top[r], d));
  // Lane l works out the scale and the reciprocal of row l mod 4 and stores the
  // scale (consecutive rows: one transaction); the others ask it.
  static_assert(FBQ_ROWS == 4, "rows a lane selects from");
  const uint32_t t01 = (l & 2) ? top[1] : top[0];
  const float mine = fb_group_scale((l & 1) ? bf16_hi(t01) : bf16_lo(t01));
  const float mine_inv = 1.0f / mine;
  if (l < FBQ_ROWS && m0 + l < M && DFK_IN_BOUNDS(g < G, 22, err))
    s[static_cast<size_t>(g) * M + m0 + l] = mine;
#pragma unroll
  for (int r = 0; r < FBQ_ROWS; ++r) {
    const FbScale f = fb_scale_of(__shfl_sync(0xffffffffu, mine, r, 16),
                                  __shfl_sync(0xffffffffu, mine_inv, r, 16));
    float v[8];
    unpack8(w[r], v);
    if (in && m0 + r < M && DFK_IN_BOUNDS(k + 8 <= K, 21, err))
      *reinterpret_cast<uint2 *>(q + static_cast<size_t>(m0 + r) * K + k) =
          make_uint2(fb_codes4(v[0], v[1], v[2], v[3], f), fb_codes4(v[4], v[5], v[6], v[7], f));
  }
}

// One CTA per row; thread t holds chunks t + T i (8 elements each, i < CPT)
// of the row in registers, so every input is read once:
//   r = bf16(x + residual)      (stored; the norm reads the rounded sum, as
//                                the next layer does)
//   v = (r / sqrt(mean r^2 + eps)) * gamma, fp32, quantised per group.
//
// LATE false (up to 1024 rows: latency counts): gamma is loaded before the
// previous kernel has finished.  LATE true (more: bandwidth counts): gamma, which
// L1 holds, is read when it is needed, so that its registers are free for
// more threads.  4096 rows of 8192: 38.5 us, 93 % of the copy rate (two chunks a
// thread and gamma early: 45 us); 2048 rows of 4096: 11.2 us against 12.4; one row
// of 4096: 1.7 us early, 2.0 late; 1024 rows: the same.
template <int CPT, bool LATE>
__global__ void __launch_bounds__(1024)
    fb_norm_kernel(const uint16_t *x, const uint16_t *res, const uint16_t *__restrict__ gamma,
                   float eps, uint16_t *res_out, uint8_t *__restrict__ q,
                   float *__restrict__ s, int M, int D, int G, unsigned *err) {
  __shared__ float s_part[32];
  const int tid = threadIdx.x, T = blockDim.x;
  const int m = blockIdx.x;
  uint4 g[CPT];
#pragma unroll
  for (int i = 0; !LATE && i < CPT; ++i) {
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
      if (res) asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(aw[j]) : "r"(bw[j]));
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
  const uint32_t rb = __float_as_uint(r);
  const float c = r == r ? __uint_as_float(rb & 0x7f800000u) : r;
  const float t = __uint_as_float((rb & 0x007fffffu) | 0x3f800000u);
  // r = c t, c a power of two and t in [1, 2): u = (a c) gamma is exact (a
  // product of two bf16 factors), and t falls out of v / s, so that the codes
  // depend on no rounding but that of max |u| / 448.  Not so where the floor or
  // an overflow to infinity parts the scales of u and of v = u t: there v itself,
  // rounded, is divided by the stored scale.
  float u[CPT][8], top[CPT];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int k = 8 * (tid + T * i);
    float w[8];
    unpack8(a[i], u[i]);
    if (LATE) {
      g[i] = make_uint4(0u, 0u, 0u, 0u);
      if (k < D) g[i] = __ldg(reinterpret_cast<const uint4 *>(gamma + k));
    }
    unpack8(g[i], w);
#pragma unroll
    for (int j = 0; j < 8; ++j) u[i][j] = (u[i][j] * c) * w[j];
    if (k >= D) {  // c may be infinite or NaN: nothing of it in the padding
#pragma unroll
      for (int j = 0; j < 8; ++j) u[i][j] = 0.f;
    }
    top[i] = group_max(abs_max8(u[i]));
  }
  // lane l mod CPT of the group's 16 works out the scale of chunk i = l mod CPT
  const int l = tid & 15, li = l % CPT;
  float mine = top[0];
#pragma unroll
  for (int i = 1; i < CPT; ++i) mine = li == i ? top[i] : mine;
  const float s_v = fb_group_scale(mine * t);
  float s_u = fb_group_scale(mine);
  const bool by_v = mine > 0.f && !(s_u > 1.17549435e-38f && s_v <= 3.402823466e38f);
  if (by_v) s_u = s_v;
  const float inv = 1.0f / s_u;
  const unsigned which = __ballot_sync(0xffffffffu, by_v) >> (tid & 16);
  if (which & 0xffffu) {
    // A loop that is not unrolled, so that the compiler makes it a branch: as
    // predicated products in every warp 4096 rows of 8192 take 39.0 us, not 38.6.
#pragma unroll 1
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        const float next = (which >> i & 1) ? u[i][0] * t : u[i][0];
#pragma unroll
        for (int e = 0; e < 7; ++e) u[i][e] = u[i][e + 1];
        u[i][7] = next;
      }
  }
  {
    const int k = 8 * (tid - l + T * li);  // the group's first element
    if (l < CPT && k < D && DFK_IN_BOUNDS(k / FB_GROUP < G && m < M, 26, err))
      s[static_cast<size_t>(k / FB_GROUP) * M + m] = s_v;
  }
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int k = 8 * (tid + T * i);
    const FbScale f = fb_scale_of(__shfl_sync(0xffffffffu, s_u, i, 16),
                                  __shfl_sync(0xffffffffu, inv, i, 16));
    if (k < D && DFK_IN_BOUNDS(k + 8 <= D && m < M, 25, err))
      *reinterpret_cast<uint2 *>(q + row + k) =
          make_uint2(fb_codes4(u[i][0], u[i][1], u[i][2], u[i][3], f),
                     fb_codes4(u[i][4], u[i][5], u[i][6], u[i][7], f));
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
  // many rows: four chunks a thread, 128 bytes on their way in each; few: as
  // many threads as there are chunks, up to the two that 1024 threads leave
  const bool late = M > 1024;
  const int cpt = late ? 4 : chunks <= 512 ? 1 : chunks <= 2048 ? 2 : 4;
  const int T = ((chunks + cpt - 1) / cpt + 31) / 32 * 32;
#define DFK_FBN(C, L) reinterpret_cast<const void *>(&fb_norm_kernel<C, L>)
  const void *fn = late       ? DFK_FBN(4, true)
                   : cpt == 1 ? DFK_FBN(1, false)
                   : cpt == 2 ? DFK_FBN(2, false)
                              : DFK_FBN(4, false);
#undef DFK_FBN
  void *args[] = {&xp, &rp, &gp, &eps, &op, &qp, &s, &M, &D, &G, &err};
  return launch_kernel(fn, dim3(M), dim3(T), 0, st, pdl, args);
}

}  // namespace dfk

// fp8_block.cuh -- block-scaled FP8: the quantisation rule every kernel of
// these operators shares, cluster helpers, and the launch interface.
//
// A vector v is stored in groups of 128 along its last dimension as E4M3
// codes q and one fp32 scale s per group:
//   a = max |v| over the group,  s = max(a / 448, 2^-126),  q = E4M3(v / s).
// 448 is E4M3's largest value, so |v / s| <= 448 (1 + 2^-23), which rounds to
// 448.  The floor 2^-126 (the smallest normal fp32) keeps s normal for tiny
// groups and non-zero for an all-zero one (codes 0).  A NaN in the group makes
// s and every code NaN; an infinity makes s infinite, its own code NaN and
// the finite elements' codes 0.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "ptx.cuh"

namespace dfk {

constexpr int FB_GROUP = 128;
constexpr float FB_E4M3_MAX = 448.f;

// max that returns NaN when either operand is NaN (fmaxf drops it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// A group's scale and the two factors of the quotient v / s.
struct FbScale {
  float s;    // the stored scale
  float inv;  // 1 / s, rounded to nearest
  float sr;   // s in the residual; 0 for an infinite s, where inv is 0 too
};

// v / b rounded to nearest, from b's correctly rounded reciprocal y and one
// residual step (Markstein, "Computation of elementary functions on the IBM
// RISC System/6000 processor", 1990; for every b but one whose mantissa is all
// ones): u = v y, u + (v - u b) y.  bf16 inputs
// often make v / s a tie between two codes, so the plain product v y, off by
// an ulp, would round a few codes in a thousand the other way.
__device__ __forceinline__ float fb_divide(float v, float b, float y) {
  const float u = v * y;
  return fmaf(fmaf(-u, b, v), y, u);
}

// The scale of a group: max(amax / 448, 2^-126), amax / 448 rounded to nearest;
// infinite for an infinite amax, NaN for a NaN.
__device__ __forceinline__ float fb_group_scale(float amax) {
  const float s = fb_divide(amax, FB_E4M3_MAX, 1.0f / FB_E4M3_MAX);
  return amax > 3.402823466e38f ? amax : max_nan(s, 1.17549435e-38f);
}

__device__ __forceinline__ FbScale fb_scale_of(float s, float inv) {
  return FbScale{s, inv, s > 3.402823466e38f ? 0.f : s};
}

__device__ __forceinline__ FbScale fb_scale(float amax) {
  const float s = fb_group_scale(amax);
  return fb_scale_of(s, 1.0f / s);
}

__device__ __forceinline__ float fb_quotient(float v, const FbScale &f) {
  return fb_divide(v, f.sr, f.inv);
}

// Four values -> four E4M3 codes, element 0 in the low byte.
__device__ __forceinline__ uint32_t fb_codes4(float v0, float v1, float v2, float v3,
                                              const FbScale &f) {
  const float u0 = fb_quotient(v0, f), u1 = fb_quotient(v1, f);
  const float u2 = fb_quotient(v2, f), u3 = fb_quotient(v3, f);
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(u0), "f"(u1), "f"(u2), "f"(u3));
  return r;
}

// SiLU(a) * u = a e^min(a, 0) / (1 + e^-|a|) * u: the denominator lies in [1, 2],
// where __fdividef is within 2 ulp.  (a / (1 + e^-a) loses all of SiLU below
// -87.3, where __fdividef returns 0 for its denominator.)  __expf is within
// 2 + 1.17 |a| ulp, far inside the 2^-4 step of a code or the 2^-8 of bf16; below
// -87.3 its result is subnormal, in steps of 2^-149.
__device__ __forceinline__ float fb_silu_mul(float a, float u) {
  const float e = __expf(-fabsf(a));
  return __fdividef(a < 0.f ? a * e : a, 1.0f + e) * u;
}

// Bounded mbarrier wait, as mbar_wait_bounded (same limits, same abort flag and
// error word), for waits that usually end within a microsecond and follow one
// another: the clock, the limit (a global load) and the abort flag are only
// looked at every 256 tries.
__device__ __forceinline__ bool fb_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag,
                                        unsigned *err) {
  unsigned long long t0 = 0, limit = 0;
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 255u) == 0) {
      if (abort_flag && *abort_flag) return false;
      const unsigned long long now = global_timer_ns();
      if (t0 == 0) {
        t0 = now;
        limit = abort_flag ? wait_limit_ns(err) : WAIT_TIMEOUT_NS;
      } else if (now - t0 > limit || it > (1u << 30)) {
        if (abort_flag) *abort_flag = 1;
        if (err) atomicOr(err, ERR_WAIT_TIMEOUT);
        return false;
      }
    }
  }
}

// As ld_act_v4, through L1 (2047 rows of 14336 quantised in 15.6 us, 16.0 without).
__device__ __forceinline__ uint4 fb_ld_v4(const void *p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// ---- thread-block clusters

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// Every thread of every CTA of the cluster; the warps converge first.
__device__ __forceinline__ void cluster_sync_all() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
               "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// As cluster_sync_all, ordering nothing: for CTAs that only wait until the others
// have read their shared memory.  A warp comes here with no read outstanding only
// if something before has used each value it read: the sums below read no column
// that is not stored, and a store cannot be issued before its operands are there.
// The release of the ordered form waits for the thread's global stores, 0.8 us at
// the end of a call.
__device__ __forceinline__ void cluster_sync_relaxed() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\t"
               "barrier.cluster.wait.aligned;" ::: "memory");
}

__device__ __forceinline__ void tensormap_prefetch(const CUtensorMap *m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// Address of the same shared-memory location in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_map(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// The cluster's shares of a token's sums (NV values of four columns, `vstep`
// bytes apart) added in rank order; at: this CTA's address of the first, the
// same in every CTA.  Four ranks' loads are on their way together.  Only the first
// nv values are read, the others are zero (cluster_sync_relaxed).
template <int NV>
__device__ __forceinline__ void fb_sum_shares(uint32_t at, uint32_t vstep, int ks, int nv,
                                              float4 (&sum)[NV]) {
#pragma unroll
  for (int v = 0; v < NV; ++v) sum[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int r0 = 0; r0 < ks; r0 += 4) {
    float4 o[4][NV];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int v = 0; v < NV; ++v)
        o[r][v] = r0 + r < ks && v < nv ? ld_cluster_f4(cluster_map(at + v * vstep, r0 + r))
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        sum[v].x += o[r][v].x;
        sum[v].y += o[r][v].y;
        sum[v].z += o[r][v].z;
        sum[v].w += o[r][v].w;
      }
  }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  return f32_to_bf16_bits(lo) | (static_cast<uint32_t>(f32_to_bf16_bits(hi)) << 16);
}

// ---- the products' arguments

struct FbMaps {
  CUtensorMap x;     // activation codes [M][K]
  CUtensorMap w[2];  // weight codes [N][K] (gate and up, or one matrix)
};

struct FbParams {
  const float *sx;     // [G][M]
  const float *sw[2];  // [ceil(N / 128)][G]
  uint16_t *y;         // [M][N] bf16, or nullptr when the output is quantised
  uint8_t *qh;         // [M][N] codes
  float *sh;           // [ceil(N / 128)][M]
  unsigned *err;
  int M, N, G;
  int stages;          // streaming kernel: ring stages
  int band;            // tensor-bound kernel: token tiles of a band
};

// bf16 output of one token's 128 weight rows (block `blk`) by a whole warp, four
// rows a lane.
template <int NMAT>
__device__ __forceinline__ void fb_emit4(const FbParams &p, int m, int blk, int lane,
                                         const float4 &a, const float4 &up) {
  const int j = blk * 128 + 4 * lane;
  float h[4] = {a.x, a.y, a.z, a.w};
  const float u[4] = {up.x, up.y, up.z, up.w};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (NMAT == 2) h[e] = fb_silu_mul(h[e], u[e]);
  uint16_t *at = p.y + static_cast<size_t>(m) * p.N + j;
  if ((p.N & 3) == 0) {
    if (j < p.N && DFK_IN_BOUNDS(j + 4 <= p.N && m < p.M, 29, p.err))
      *reinterpret_cast<uint2 *>(at) =
          make_uint2(pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (j + e < p.N && DFK_IN_BOUNDS(m < p.M, 30, p.err)) at[e] = f32_to_bf16_bits(h[e]);
  }
}

// Quantised output of a gated product, one token by a whole warp.
__device__ __forceinline__ void fb_emit4_codes(const FbParams &p, int m, int blk, int lane,
                                               const float4 &a, const float4 &up) {
  const int j = blk * 128 + 4 * lane;
  float h[4] = {a.x, a.y, a.z, a.w};
  const float u[4] = {up.x, up.y, up.z, up.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    h[e] = fb_silu_mul(h[e], u[e]);
    if (j + e >= p.N) h[e] = 0.f;
  }
  float mx = max_nan(max_nan(fabsf(h[0]), fabsf(h[1])), max_nan(fabsf(h[2]), fabsf(h[3])));
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, d));
  const FbScale f = fb_scale(mx);
  if (j < p.N && DFK_IN_BOUNDS(j + 4 <= p.N && m < p.M, 35, p.err))
    *reinterpret_cast<uint32_t *>(p.qh + static_cast<size_t>(m) * p.N + j) =
        fb_codes4(h[0], h[1], h[2], h[3], f);
  if (lane == 0) p.sh[static_cast<size_t>(blk) * p.M + m] = f.s;
}

// Quantised output of a gated product: nt tokens (the first is token m0), weight
// rows of block `blk` (one group), summed over the cluster's CTAs in rank order.
// at: shared-memory address of token 0's 128 gate sums, `tstep` bytes from token to
// token, `mstep` from a token's gate sums to its up sums.  Eight lanes take a
// token, sixteen rows each; this warp is the w-th of nw in CTA `rank`.  Rows at or
// past N, which are not stored, are not read (cluster_sync_relaxed).  (A token a
// turn and warp: 64 tokens took 3 us, each a chain of loads, SiLU, five shuffles,
// two reciprocals.)
__device__ __forceinline__ void fb_emit_codes(const FbParams &p, uint32_t at, uint32_t tstep,
                                              uint32_t mstep, int nt, int m0, int blk, int w,
                                              int nw, int rank, int ks, int lane) {
  const int l = lane & 7;
  for (int quad = rank * nw + w; 4 * quad < nt; quad += nw * ks) {
    const int n = 4 * quad + (lane >> 3);
    const uint32_t mine = at + static_cast<uint32_t>(min(n, nt - 1)) * tstep + 16 * l;
    const int j = blk * 128 + 4 * l;  // and 32 further on for each i; N % 16 == 0
    float h[16], u[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) h[i] = u[i] = 0.f;
    for (int r = 0; r < ks; ++r) {
      const uint32_t src = cluster_map(mine, ks == 1 ? rank : r);
      float4 g[4], v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        g[i] = v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j + 32 * i < p.N) {
          g[i] = ld_cluster_f4(src + 128 * i);
          v[i] = ld_cluster_f4(src + 128 * i + mstep);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[4 * i] += g[i].x;
        h[4 * i + 1] += g[i].y;
        h[4 * i + 2] += g[i].z;
        h[4 * i + 3] += g[i].w;
        u[4 * i] += v[i].x;
        u[4 * i + 1] += v[i].y;
        u[4 * i + 2] += v[i].z;
        u[4 * i + 3] += v[i].w;
      }
    }
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      h[i] = fb_silu_mul(h[i], u[i]);
      mx = max_nan(mx, fabsf(h[i]));
    }
#pragma unroll
    for (int d = 4; d >= 1; d >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    const FbScale f = fb_scale(mx);
    if (n < nt) {
      uint8_t *q = p.qh + static_cast<size_t>(m0 + n) * p.N + j;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (j + 32 * i < p.N && DFK_IN_BOUNDS(j + 32 * i + 4 <= p.N && m0 + n < p.M, 28, p.err))
          *reinterpret_cast<uint32_t *>(q + 32 * i) =
              fb_codes4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3], f);
      if (l == 0) p.sh[static_cast<size_t>(blk) * p.M + m0 + n] = f.s;
    }
  }
}

// kernels of fp8_block_quant.cu / fp8_block_small.cu
cudaError_t launch_fb_quant(const void *x, void *q, float *s, int M, int K, unsigned *err,
                            cudaStream_t st, bool pdl);
cudaError_t launch_fb_norm(const void *x, const void *res, const void *gamma, float eps,
                           void *res_out, void *q, float *s, int M, int D, unsigned *err,
                           cudaStream_t st, bool pdl);
constexpr int FB_NORM_MAX_D = 32768  /* 4 chunks of 8 in each of 1024 threads */;

const void *fb_small_kernel(int nmat, int bn);
int fb_small_threads(int nmat, int bn);
int fb_small_smem(int nmat, int bn, int stages);
int fb_small_min_stages(int nmat, int bn);

// fp8_block_large.cu: tiles of 256 tokens by pairs of CTAs (`pair`), or of 128 tokens
// by CTAs of their own, `ks` of them to a tile
const void *fb_large_kernel_fn(bool gate, bool pair);
int fb_large_weight_box(bool pair);  // rows of the weights' TMA box
cudaError_t launch_fb_large(bool gate, bool pair, int ks, const FbMaps &maps, const FbParams &p,
                            int sms, cudaStream_t st, bool pdl);

}  // namespace dfk

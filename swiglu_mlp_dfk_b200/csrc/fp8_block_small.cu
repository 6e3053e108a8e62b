// fp8_block_small.cu -- block-scaled FP8 products for few tokens: weight
// streaming.  y[m][n] = sum_kb s_x[kb][m] s_w[n/128][kb] P_kb[n][m], where
// P_kb is the product of the codes over one group of 128, exact products
// summed in fp32 by the E4M3 tensor-core MMA.
//
// One CTA owns 128 weight rows (one scale block of each matrix: the MMA's M)
// and BN tokens (its N), over all groups or, in a cluster of `ks` CTAs, over a
// share of them.  A TMA ring carries one group per stage: 128 x 128 codes of
// each matrix and BN x 128 activation codes.  The accumulator of a group is
// read back from TMEM while the tensor core fills the other one (two TMEM
// buffers), scaled by s_x s_w and added in fp32 registers: the scales change
// every 128 steps of k, so no sum can stay in TMEM across groups.  The CTAs
// of a cluster add their shares in rank order through distributed shared
// memory: no scratch memory, no atomics, the same bits every time.
#include "fp8_block.cuh"
#include "tc_ptx.cuh"
#include "tf8mma_engine.cuh"

namespace dfk {

constexpr int FBS_WTILE = 128 * 128;
constexpr int FBS_PRE = 4;         // groups whose scales are loaded ahead

template <int NMAT, int BN>
struct FbsShape {
  // epilogue warps: one for each TMEM lane quarter, two where four would have
  // 64 sums a thread or more (4096 x 14336 gated: 64 tokens 27.3 us with four,
  // 23.5 with eight; 32 tokens 22.8 and 22.0)
  static constexpr int warps = NMAT * BN >= 64 ? 8 : 4;
  static constexpr int threads = 64 + 32 * warps;  // TMA warp, MMA warp
  static constexpr int tokens = BN * 4 / warps;    // of one epilogue thread
  static constexpr int stage_bytes = NMAT * FBS_WTILE + BN * 128;
  static constexpr int acc_cols = NMAT * BN;       // one TMEM buffer
  static constexpr int tmem_cols = 2 * acc_cols < 32 ? 32 : 2 * acc_cols;
  static constexpr int comb_floats = warps * 2 * NMAT * tokens;  // per warp, two groups
  static constexpr int part_bytes = NMAT * BN * 128 * 4;
  static constexpr int min_stages =
      part_bytes > 2 * stage_bytes ? (part_bytes + stage_bytes - 1) / stage_bytes : 2;
};

// 16 or 32 TMEM columns of this warp's lanes; the values may be used after
// tmem_ld_wait.
template <int N>
__device__ __forceinline__ void tmem_cols(uint32_t taddr, float (&d)[N]) {
  static_assert(N == 16 || N == 32, "columns a load");
  if constexpr (N == 16) {
    tmem_ld_32x32b_x16(taddr, d);
  } else {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) d[i] = __uint_as_float(r[i]);
  }
}

template <int NMAT, int BN>
__global__ void __launch_bounds__(FbsShape<NMAT, BN>::threads)
    fb_small_kernel_t(const __grid_constant__ FbMaps maps, const FbParams p) {
  using Sh = FbsShape<NMAT, BN>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw_addr = smem_addr(smem_raw);
  uint8_t *smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const uint32_t sbase = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = p.stages;

  float *s_comb = reinterpret_cast<float *>(smem + static_cast<size_t>(S) * Sh::stage_bytes);
  uint64_t *fullb = reinterpret_cast<uint64_t *>(s_comb + Sh::comb_floats);
  uint64_t *empty = fullb + S;
  uint64_t *accfull = empty + S;  // [2]
  uint64_t *accempty = accfull + 2;
  uint64_t *done = accempty + 2;
  volatile int *s_abort = reinterpret_cast<volatile int *>(done + 1);
  int *s_issued = reinterpret_cast<int *>(done + 1) + 1;
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(done + 1) + 2;

  // clusters of ks consecutive blocks share a row block
  uint32_t ks;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ks));
  const uint32_t rank = cluster_rank();
  const int blk = blockIdx.x / ks;
  const int j0 = blk * 128, n0 = blockIdx.y * BN;
  const int kb0 = static_cast<int>(static_cast<long long>(rank) * p.G / ks);
  const int kb1 = static_cast<int>(static_cast<long long>(rank + 1) * p.G / ks);
  const int nkb = kb1 - kb0;

  // Thread 0 sets the barriers up and at once sends for the weights of the first
  // stages (before the dependency on the previous kernel; the activation codes
  // follow after it).
  const uint64_t pol_w = gridDim.y > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
  const int S0 = min(S, nkb);
  auto load_w = [&](int i, int st) {
    uint8_t *sb = smem + st * Sh::stage_bytes;
    mbar_arrive_expect_tx(&fullb[st], Sh::stage_bytes);
#pragma unroll
    for (int m = 0; m < NMAT; ++m)
      tma_load_2d(sb + m * FBS_WTILE, &maps.w[m], &fullb[st], (kb0 + i) * 128, j0, pol_w);
  };
  if (tid == 0) {
#pragma unroll
    for (int m = 0; m < NMAT; ++m) tensormap_prefetch(&maps.w[m]);
    tensormap_prefetch(&maps.x);
    for (int s = 0; s < S; ++s) {
      mbar_init(&fullb[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&accfull[s], 1);
      mbar_init(&accempty[s], Sh::warps);
    }
    mbar_init(done, 1);
    *s_abort = 0;
    *s_issued = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    for (int i = 0; i < S0; ++i) load_w(i, i);
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, Sh::tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  pdl_launch_dependents();

  if (warp == 0) {
    // ---- TMA
    if (lane == 0) {
      const uint64_t pol_x = l2_policy_evict_normal();
      auto load_x = [&](int i, int st) {
        tma_load_2d(smem + st * Sh::stage_bytes + NMAT * FBS_WTILE, &maps.x, &fullb[st],
                    (kb0 + i) * 128, n0, pol_x);
      };
      pdl_wait();
      for (int i = 0; i < S0; ++i) load_x(i, i);
      int issued = S0, st = 0;
      uint32_t ph = 0;  // of the stage's last use; stages and phases are counted along:
                        // S is no constant, and a division costs as much as a wait
      for (int i = S0; i < nkb; ++i) {
        if (!fb_wait(&empty[st], ph, s_abort, p.err)) break;
        load_w(i, st);
        load_x(i, st);
        issued = i + 1;
        if (++st == S) {
          st = 0;
          ph ^= 1u;
        }
      }
      *s_issued = issued;
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---- MMA: 4 instructions of K = 32 per matrix and group
    const uint32_t leader = elect_one_sync();
    const uint32_t idesc = umma_idesc_e4m3_f32(128, BN);
    const uint64_t desc0 = umma_desc_sw128(sbase);
    int st = 0;
    uint32_t ph = 0;
    for (int i = 0; i < nkb; ++i) {
      const int ab = i & 1;
      bool ok = i < 2 || fb_wait(&accempty[ab], ((i >> 1) - 1) & 1, s_abort, p.err);
      ok = ok && fb_wait(&fullb[st], ph, s_abort, p.err);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const uint64_t ds = desc0 + (static_cast<uint32_t>(st * Sh::stage_bytes) >> 4);
      const uint64_t bx = ds + (static_cast<uint32_t>(NMAT * FBS_WTILE) >> 4);
#pragma unroll
      for (int m = 0; m < NMAT; ++m)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          if (leader)
            umma_e4m3(tmem + static_cast<uint32_t>(ab * Sh::acc_cols + m * BN),
                      ds + m * (FBS_WTILE >> 4) + 2 * kk, bx + 2 * kk, idesc, kk > 0 ? 1u : 0u);
      if (leader) {
        umma_commit(&empty[st]);
        umma_commit(&accfull[ab]);
      }
      __syncwarp();
      if (++st == S) {
        st = 0;
        ph ^= 1u;
      }
    }
    if (leader) umma_commit(done);
    __syncwarp();
  } else {
    // ---- epilogue warps: TMEM lane quarter = warp mod 4, a share of the tokens
    const int ew = warp - 2, q = warp & 3;
    const int row = 32 * q + lane;
    constexpr int TN = Sh::tokens;
    const int t0 = (ew >> 2) * TN;  // the warp's first token
    const uint32_t base = tmem + (static_cast<uint32_t>(32 * q) << 16) + t0;
    constexpr int SL = (TN + 31) / 32;  // tokens a lane loads scales for
    float *comb = s_comb + ew * 2 * NMAT * TN;
    uint64_t acc[NMAT][TN / 2];  // pairs of tokens
#pragma unroll
    for (int m = 0; m < NMAT; ++m)
#pragma unroll
      for (int n = 0; n < TN / 2; ++n) acc[m][n] = 0ull;
    float psx[FBS_PRE][SL], psw[FBS_PRE][NMAT];
    pdl_wait();  // s_x comes from the previous kernel
    auto fetch = [&](int i, float (&sx)[SL], float (&sw)[NMAT]) {
      const int kb = kb0 + i;
#pragma unroll
      for (int m = 0; m < NMAT; ++m)
        sw[m] = i < nkb ? __ldg(p.sw[m] + static_cast<size_t>(blk) * p.G + kb) : 0.f;
#pragma unroll
      for (int e = 0; e < SL; ++e) {
        const int n = n0 + t0 + lane + 32 * e;
        sx[e] = 0.f;
        if (i < nkb && lane + 32 * e < TN && n < p.M && DFK_IN_BOUNDS(kb < p.G, 27, p.err))
          sx[e] = ld_act_f32(p.sx + static_cast<size_t>(kb) * p.M + n);
      }
    };
#pragma unroll
    for (int u = 0; u < FBS_PRE; ++u) fetch(u, psx[u], psw[u]);
    bool go = true;
    for (int i0 = 0; go && i0 < nkb; i0 += FBS_PRE) {
#pragma unroll
      for (int u = 0; u < FBS_PRE; ++u) {
        const int i = i0 + u;
        if (go && i < nkb) {
          const int ab = u & 1;  // FBS_PRE is even: the same as i & 1
          // this group's s_x s_w, one per token, for the whole warp
          float *cb = comb + ab * NMAT * TN;
#pragma unroll
          for (int m = 0; m < NMAT; ++m)
#pragma unroll
            for (int e = 0; e < SL; ++e)
              if (TN >= 32 || lane < TN) cb[m * TN + lane + 32 * e] = psx[u][e] * psw[u][m];
          fetch(i + FBS_PRE, psx[u], psw[u]);
          __syncwarp();
          go = __all_sync(0xffffffffu, fb_wait(&accfull[ab], (i >> 1) & 1, s_abort,
                                                         p.err));
          if (go) {
            tc_fence_after();
            constexpr int CH = TN < 32 ? TN : 32;
#pragma unroll
            for (int c = 0; c < TN; c += CH) {
              float d[NMAT][CH];
#pragma unroll
              for (int m = 0; m < NMAT; ++m)
                tmem_cols<CH>(base + ab * Sh::acc_cols + m * BN + c, d[m]);
              tmem_ld_wait();
#pragma unroll
              for (int m = 0; m < NMAT; ++m)
#pragma unroll
                for (int e = 0; e < CH; e += 4) {
                  const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(cb + m * TN + c + e);
                  uint64_t *s = &acc[m][(c + e) / 2];
                  s[0] = fma_f32x2(pack_f32x2(d[m][e], d[m][e + 1]), w.x, s[0]);
                  s[1] = fma_f32x2(pack_f32x2(d[m][e + 2], d[m][e + 3]), w.y, s[1]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&accempty[ab]);
          }
        }
      }
    }
    // every MMA has read its stage by now: the ring holds the partial sums
    // [matrix][token][row]
    float *part = reinterpret_cast<float *>(smem);
    if (go)
#pragma unroll
      for (int m = 0; m < NMAT; ++m)
#pragma unroll
        for (int n = 0; n < TN / 2; ++n) {
          float lo, hi;
          unpack_f32x2(acc[m][n], lo, hi);
          part[(m * BN + t0 + 2 * n) * 128 + row] = lo;
          part[(m * BN + t0 + 2 * n + 1) * 128 + row] = hi;
        }
  }

  // TMEM is released and the copies in flight are waited for before the
  // cluster meets (after an abort; normally all have been consumed)
  __syncthreads();
  if (warp == 1) {
    if (lane == 0) fb_wait(done, 0, nullptr, p.err);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, Sh::tmem_cols);
  }
  if (tid == 0 && *s_abort) {
    const int issued = *s_issued;
    for (int st = 0; st < S; ++st) {
      int last = -1;
      for (int i = issued - 1; i >= 0 && i >= issued - S; --i)
        if (i % S == st) { last = i; break; }
      if (last >= 0) fb_wait(&fullb[st], (last / S) & 1, nullptr, p.err);
    }
  }
  __syncwarp();
  if (ks > 1) cluster_sync_all();
  if (warp >= 2 && !*s_abort) {
    // one token per warp and turn, spread over the cluster's CTAs; lane l
    // takes rows 4 l .. 4 l + 3
    const int nt = min(BN, p.M - n0);
    if (NMAT == 2 && p.y == nullptr) {
      fb_emit_codes(p, sbase, 512, BN * 512, nt, n0, blk, warp - 2, Sh::warps, rank, ks, lane);
    } else if (ks == 1) {
      // four tokens' sums in registers at a time: one after the other, a round
      // trip each, cost up to 2 us
      for (int n = warp - 2; n < nt; n += 4 * Sh::warps) {
        float4 a[4][NMAT];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int m = 0; m < NMAT; ++m)
            a[u][m] = *reinterpret_cast<const float4 *>(
                smem + ((m * BN + min(n + u * Sh::warps, BN - 1)) * 128 + 4 * lane) * 4);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (n + u * Sh::warps < nt)
            fb_emit4<NMAT>(p, n0 + n + u * Sh::warps, blk, lane, a[u][0], a[u][NMAT - 1]);
      }
    } else {
      for (int n = rank * Sh::warps + (warp - 2); n < nt; n += Sh::warps * ks) {
        float4 a[NMAT];
        fb_sum_shares<NMAT>(sbase + static_cast<uint32_t>((n * 128 + 4 * lane) * 4), BN * 512, ks,
                            NMAT, a);
        fb_emit4<NMAT>(p, n0 + n, blk, lane, a[0], a[NMAT - 1]);
      }
    }
  }
  __syncwarp();
  if (ks > 1) cluster_sync_relaxed();  // no CTA leaves while its sums are being read
}

template <int NMAT, int BN>
static int smem_of(int stages) {
  using Sh = FbsShape<NMAT, BN>;
  const int ring = stages * Sh::stage_bytes;
  return 1024 + ring + Sh::comb_floats * 4 + (2 * stages + 5) * 8 + 16;
}

#define DFK_FBS_PICK(expr)                             \
  (nmat == 1 ? (bn == 16   ? expr(1, 16)                \
                : bn == 32 ? expr(1, 32) : expr(1, 64)) \
             : (bn == 16   ? expr(2, 16)                \
                : bn == 32 ? expr(2, 32) : expr(2, 64)))

const void *fb_small_kernel(int nmat, int bn) {
#define DFK_FBS_FN(NM, B) reinterpret_cast<const void *>(&fb_small_kernel_t<NM, B>)
  return DFK_FBS_PICK(DFK_FBS_FN);
#undef DFK_FBS_FN
}

int fb_small_threads(int nmat, int bn) {
#define DFK_FBS_TH(NM, B) FbsShape<NM, B>::threads
  return DFK_FBS_PICK(DFK_FBS_TH);
#undef DFK_FBS_TH
}

int fb_small_min_stages(int nmat, int bn) {
#define DFK_FBS_MS(NM, B) FbsShape<NM, B>::min_stages
  return DFK_FBS_PICK(DFK_FBS_MS);
#undef DFK_FBS_MS
}

int fb_small_smem(int nmat, int bn, int stages) {
#define DFK_FBS_SM(NM, B) smem_of<NM, B>(stages)
  return DFK_FBS_PICK(DFK_FBS_SM);
#undef DFK_FBS_SM
}

}  // namespace dfk

// fp8_block_large.cu -- block-scaled FP8 products for many tokens (prompts):
// bound by the E4M3 tensor-core MMA and, at length, by the power limit.
//
//   y[m][n] = sum_kb s_x[kb][m] s_w[n/128][kb] P_kb[m][n],
// P_kb the product of the codes over one group of 128.  Two forms of one kernel:
//
// PAIR: two CTAs (cluster of 2, cta_group::2) own a tile of 256 tokens (the MMA's
// M, 128 in each CTA's TMEM lanes) x 256 weight rows, of which each CTA brings
// 128: 32 KB of codes per CTA and group feed 512 tensor-core cycles.  For the
// gated product CTA 0 brings 128 gate rows and CTA 1 the matching 128 up rows, so
// each CTA holds both halves of 128 columns of h: one group of the quantised
// output.  One persistent pair per two SMs walks the tiles in bands of token
// tiles, so that the tiles in flight share operands in L2.
//
// Single: a CTA owns 128 tokens x 256 weight rows (48 KB per group); where there
// are few tiles, clusters of 2 or 4 CTAs share a tile's groups and add their sums
// in rank order through distributed shared memory.
//
// The scales change with every group, so a group's sums leave TMEM, are
// multiplied by s_x s_w and added to fp32 registers: 128 sums in each of 256
// epilogue threads, one token per thread, two at a time (fma.rn.f32x2).  TMEM
// holds two groups in two halves of 128 columns each, every half with barriers of
// its own: four epilogue warps empty one half while the tensor core fills
// another.  Two warps of their own work out s_x s_w and report through the same
// barrier as the MMA.
//
// Measured (B200): 4096 tokens, K = 4096, gated, d_ff = 14336: 425 us in a burst
// (2.27 PFLOP/s), 490 us for seconds on end (1.97, SM clock 1.4 GHz under the
// 1000 W limit); K = 14336, N = 4096: 214 and 254 us.  Stamps of the SM clock, which
// stands at 1.5 GHz from the first of such calls on: 650 to 670 cycles a group, of
// which the MMA needs 512, and 4400 cycles for a gated tile's output (3900 plain):
// 17 % of the gated call (25 tiles of 32 groups a pair), 5 % of the plain one (4 of
// 112).  On the way: one barrier per group instead of per half 524 us; loads of 32
// TMEM columns instead of 16 680 cycles a group in place of 480 in a test of the loop
// alone (the allocator copies registers); sixteen epilogue warps of 64 sums no faster;
// single CTAs in place of pairs 14 % slower.
#include <algorithm>

#include "fp8_block.cuh"
#include "launch_util.h"
#include "tc_ptx.cuh"
#include "tf8mma_engine.cuh"

namespace dfk {

constexpr int FBL_THREADS = 384;   // TMA, MMA and two scale warps; eight epilogue warps
// Registers a thread: 384 x 168 at launch, then 56 for the first warpgroup and
// 224 for the two epilogue warpgroups (56 + 2 x 224 = 3 x 168).
constexpr int FBL_REGS_IO = 56, FBL_REGS_EPI = 224;
constexpr int FBL_HALF = 128 * 128;           // bytes of one operand's half tile
constexpr int FBL_RING = 12 * FBL_HALF;       // six stages of a pair, four of a single CTA
constexpr int FBL_MAX_STAGES = 6;
constexpr int FBL_PART_ROW = 1040;            // a token's 256 partial sums and 16 bytes
constexpr int FBL_AHEAD = 8;       // groups whose scales are on the way (a power of two)
constexpr int FBL_COMB = 4;        // groups whose s_x s_w are ready (a power of two)
// A band of token tiles is as many as keep its activation codes, which every column
// tile reads again, to a quarter of L2: the weights then come from HBM once a band.
// Sustained, 8192 tokens, K = 4096, gated 8192: 576 us in bands of 8, 558 of 32;
// K = N = 8192: 555 of 8, 553 of 16, 617 of 32.
constexpr long long FBL_BAND_BYTES = 32 << 20;

constexpr int FBL_OFF_OUT = FBL_RING;                      // 8 warps x 2 KB: output rows
constexpr int FBL_OFF_SX = FBL_OFF_OUT + 8 * 2048;         // [AHEAD][128] s_x
constexpr int FBL_OFF_SW = FBL_OFF_SX + FBL_AHEAD * 512;   // [AHEAD][2 warps][2] s_w
constexpr int FBL_OFF_COMB = FBL_OFF_SW + FBL_AHEAD * 16;  // [COMB][2][128] s_x s_w
constexpr int FBL_OFF_MAX = FBL_OFF_COMB + FBL_COMB * 1024;  // [2 tiles][2][128] row maxima
constexpr int FBL_OFF_BAR = FBL_OFF_MAX + 2048;
constexpr int FBL_BARS = 2 * FBL_MAX_STAGES + 13;
constexpr int FBL_SMEM = 1024 + FBL_OFF_BAR + FBL_BARS * 8 + 16;

// ---- cta_group::2 forms

__device__ __forceinline__ void tmem_alloc_pair(uint32_t *slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_addr(slot)),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}

// D (both CTAs' TMEM) (+)= A B^T; the descriptors' offsets hold in both CTAs.
__device__ __forceinline__ void umma_e4m3_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                               uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrive on the barrier at this offset in both CTAs once the MMAs issued so
// far have completed.
__device__ __forceinline__ void umma_commit_pair(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(smem_addr(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// Tile copy into this CTA's shared memory, counted on a barrier of the pair
// (`bar`: a shared::cluster address, the leader's).
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map, uint32_t bar,
                                                 int c0, int c1, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2.L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "l"(policy)
      : "memory");
}

// Arrive on a barrier of the pair (a shared::cluster address).  Release at CTA
// scope: what it hands over are TMEM reads, ordered by tcgen05.wait::ld and
// the fence before it.  A release at cluster scope waits for the thread's
// global copies in flight: 1500 cycles per group.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}

// 16 TMEM columns of this warp's lanes; the values may be used after
// tmem_wait16, which takes them as operands.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// Whether the phase has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const float *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Tile number -> (token tile, column tile): bands of token tiles, inside a band
// column tile by column tile.
struct FblTiles {
  int tm, tn, band;
  __device__ __forceinline__ int count() const { return tm * tn; }
  __device__ __forceinline__ void at(int t, int &m, int &n) const {
    const int b = t / (band * tn), r = t - b * band * tn;
    const int h = min(band, tm - b * band);
    n = r / h;
    m = b * band + (r - n * h);
  }
};

// A warp's output goes to global memory through 2 KB of shared memory, so that
// whole 32-byte sectors of a row are written together: 32 rows (lane = row) of 64
// bytes, chunks of 16 bytes swizzled so that neither side meets a bank twice.
__device__ __forceinline__ uint8_t *fbl_chunk(uint8_t *buf, int r, int c) {
  return buf + r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ void fbl_stage(uint8_t *buf, int lane, const uint32_t (&w)[16]) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint4 *>(fbl_chunk(buf, lane, c)) =
        make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  __syncwarp();
}

// The staged rows m0 .. m0 + 31, columns n0 .. n0 + 31 of y: 16 bytes a lane where
// the rows of y are aligned for it, else neighbouring lanes store neighbouring
// pairs (N even) or elements of one row.
__device__ __forceinline__ void fbl_store_bf16(const FbParams &p, uint8_t *buf, int lane, int m0,
                                               int n0) {
  if ((p.N & 7) == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2), c = lane & 3, m = m0 + r, col = n0 + 8 * c;
      const uint4 v = *reinterpret_cast<const uint4 *>(fbl_chunk(buf, r, c));
      if (m < p.M && col < p.N && DFK_IN_BOUNDS(col + 8 <= p.N, 31, p.err))
        *reinterpret_cast<uint4 *>(p.y + static_cast<size_t>(m) * p.N + col) = v;
    }
  } else if ((p.N & 1) == 0) {
    const int e = 2 * (lane & 15), col = n0 + e;
#pragma unroll 4
    for (int r = lane >> 4; r < 32; r += 2) {
      const uint32_t v =
          *reinterpret_cast<const uint32_t *>(fbl_chunk(buf, r, e >> 3) + 2 * (e & 7));
      if (m0 + r < p.M && col < p.N && DFK_IN_BOUNDS(col + 2 <= p.N, 36, p.err))
        *reinterpret_cast<uint32_t *>(p.y + static_cast<size_t>(m0 + r) * p.N + col) = v;
    }
  } else {
    const int col = n0 + lane;
#pragma unroll 4
    for (int r = 0; r < 32; ++r) {
      const uint16_t v =
          *reinterpret_cast<const uint16_t *>(fbl_chunk(buf, r, lane >> 3) + 2 * (lane & 7));
      if (m0 + r < p.M && col < p.N) p.y[static_cast<size_t>(m0 + r) * p.N + col] = v;
    }
  }
  __syncwarp();
}

template <bool GATE, bool PAIR>
__global__ void __launch_bounds__(FBL_THREADS, 1)
    fb_large_kernel(const __grid_constant__ FbMaps maps, const FbParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw_addr = smem_addr(smem_raw);
  uint8_t *smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const uint32_t sbase = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int STAGE = (PAIR ? 2 : 3) * FBL_HALF, S = FBL_RING / STAGE;

  uint64_t *fullb = reinterpret_cast<uint64_t *>(smem + FBL_OFF_BAR);  // the leader's count
  uint64_t *empty = fullb + S;
  uint64_t *accfull = empty + S;    // [2 buffers][2 halves]
  uint64_t *accempty = accfull + 4; // [2][2], the leader's count
  uint64_t *maxfull = accempty + 4; // [4] row maxima of both halves written, per lane quarter
  uint64_t *done = maxfull + 4;
  volatile int *s_abort = reinterpret_cast<volatile int *>(done + 1);
  int *s_issued = reinterpret_cast<int *>(done + 1) + 1;
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(done + 1) + 2;

  const uint32_t rank = cluster_rank();
  uint32_t csize;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(csize));
  const int unit = blockIdx.x / csize, nunits = gridDim.x / csize;
  // a single CTA's share of the groups (PAIR: all; its CTAs share the tokens)
  const int ks = PAIR ? 1 : static_cast<int>(csize), kr = PAIR ? 0 : static_cast<int>(rank);
  const int kb0 = static_cast<int>(static_cast<long long>(kr) * p.G / ks);
  const int nkb = static_cast<int>(static_cast<long long>(kr + 1) * p.G / ks) - kb0;
  constexpr int TM = PAIR ? 256 : 128;             // tokens of a tile
  const int m_cta = PAIR ? static_cast<int>(rank) * 128 : 0;  // this CTA's first in it
  const uint32_t lead = PAIR ? 0u : rank;          // the CTA that issues the MMAs
  const int NB = (p.N + 127) / 128;  // scale blocks along the weight rows
  const FblTiles tiles{(p.M + TM - 1) / TM, GATE ? NB : (p.N + 255) / 256, p.band};
  const int ntiles = tiles.count();
  const int total = (ntiles - unit + nunits - 1) / nunits * nkb;  // groups of this CTA

  if (tid == 0) {
    tensormap_prefetch(&maps.w[0]);
    if (GATE) tensormap_prefetch(&maps.w[1]);
    tensormap_prefetch(&maps.x);
    for (int s = 0; s < S; ++s) {
      mbar_init(&fullb[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&accfull[s], 3);   // the MMAs of a group's half and both scale warps
      mbar_init(&accempty[s], PAIR ? 8 : 4);  // four epilogue warps of each CTA
    }
    for (int s = 0; s < 4; ++s) mbar_init(&maxfull[s], 2);
    mbar_init(done, 1);
    *s_abort = 0;
    *s_issued = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(s_tmem, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(s_tmem, 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist before either is signalled
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  pdl_launch_dependents();

  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FBL_REGS_IO));
  if (warp == 0) {
    // ---- TMA: this CTA's 128 tokens and, of every group, its 128 weight rows
    // (PAIR) or all 256: 64 rows of each half after the other
    if (lane == 0) {
      const uint64_t pol = l2_policy_evict_normal();
      auto load_w = [&](int kb, int st, int tn) {
        uint8_t *sb = smem + st * STAGE + FBL_HALF;
        if constexpr (PAIR) {
          if (rank == 0) mbar_arrive_expect_tx(&fullb[st], 2 * STAGE);
          const CUtensorMap *wmap = GATE && rank ? &maps.w[1] : &maps.w[0];
          const int wrow = GATE ? tn * 128 : tn * 256 + static_cast<int>(rank) * 128;
          tma_load_2d_pair(sb, wmap, cluster_map(smem_addr(&fullb[st]), 0), kb * 128, wrow, pol);
        } else {
          mbar_arrive_expect_tx(&fullb[st], STAGE);
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // half i / 2, matrix or 128-row block i % 2
            const int wrow = (GATE ? tn * 128 : tn * 256 + 128 * (i & 1)) + 64 * (i >> 1);
            tma_load_2d(sb + i * (FBL_HALF / 2), &maps.w[GATE ? i & 1 : 0], &fullb[st], kb * 128,
                        wrow, pol);
          }
        }
      };
      // the first stages' weights, before the dependency on the previous kernel (a
      // layer of norm, gate/up and down, 96 tokens, 4096 x 14336: 49.5 -> 48.9 us)
      const int early = min(S, nkb);
      int tm, tn;
      tiles.at(unit, tm, tn);
      for (int i = 0; i < early; ++i) load_w(kb0 + i, i, tn);
      pdl_wait();
      int it = 0, st = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = unit; ok && t < ntiles; t += nunits) {
        tiles.at(t, tm, tn);
        const int mrow = tm * TM + m_cta;
        for (int kb = kb0; kb < kb0 + nkb; ++kb, ++it) {
          if (it >= S && !fb_wait(&empty[st], ph ^ 1u, s_abort, p.err)) {
            ok = false;
            break;
          }
          if (it >= early) load_w(kb, st, tn);
          if constexpr (PAIR)
            tma_load_2d_pair(smem + st * STAGE, &maps.x, cluster_map(smem_addr(&fullb[st]), 0),
                             kb * 128, mrow, pol);
          else
            tma_load_2d(smem + st * STAGE, &maps.x, &fullb[st], kb * 128, mrow, pol);
          if (++st == S) {
            st = 0;
            ph ^= 1u;
          }
        }
      }
      *s_issued = it;
      // the last stages' releases have arrived before this CTA may leave
      for (int i = max(0, it - S); ok && i < it; ++i)
        ok = fb_wait(&empty[i % S], (i / S) & 1, s_abort, p.err);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---- MMA (PAIR: CTA 0 for both): per half 4 instructions of K = 32
    const uint32_t leader = elect_one_sync();
    if (rank == lead) {
      const uint32_t idesc = umma_idesc_e4m3_f32(PAIR ? 256 : 128, 128);
      const uint64_t desc0 = umma_desc_sw128(sbase);
      // rows 64 h .. 64 h + 63 of both 128-row halves of the weights
      constexpr uint32_t HALF_ENC = (PAIR ? FBL_HALF / 2 : FBL_HALF) >> 4;
      auto commit = [&](uint64_t *bar) {
        if constexpr (PAIR) umma_commit_pair(bar);
        else umma_commit(bar);
      };
      int st = 0;
      uint32_t ph = 0;
      for (int it = 0; it < total; ++it) {
        const int ab = it & 1;
        bool ok = fb_wait(&fullb[st], ph, s_abort, p.err);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        const uint64_t da = desc0 + (static_cast<uint32_t>(st * STAGE) >> 4);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ok = it < 2 || fb_wait(&accempty[2 * ab + h], ((it >> 1) - 1) & 1, s_abort, p.err);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint64_t db = da + (FBL_HALF >> 4) + h * HALF_ENC;
          const uint32_t d = tmem + static_cast<uint32_t>(ab * 256 + h * 128);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            if (leader) {
              if constexpr (PAIR)
                umma_e4m3_pair(d, da + 2 * kk, db + 2 * kk, idesc, kk > 0 ? 1u : 0u);
              else
                umma_e4m3(d, da + 2 * kk, db + 2 * kk, idesc, kk > 0 ? 1u : 0u);
            }
          if (leader) commit(&accfull[2 * ab + h]);
          __syncwarp();
        }
        if (!ok) break;
        if (leader) commit(&empty[st]);
        __syncwarp();
        if (++st == S) {
          st = 0;
          ph ^= 1u;
        }
      }
      if (leader) commit(done);
      __syncwarp();
    }
  } else if (warp < 4) {
    // ---- scales: the product s_x s_w of every token and both halves of the
    // tile's columns (gated: both matrices), a few groups ahead of the epilogue.
    // A warp takes 64 tokens; raw scales are copied FBL_AHEAD groups ahead.
    const int w = warp - 2, row = 64 * w + lane;
    float *s_sx = reinterpret_cast<float *>(smem + FBL_OFF_SX);
    float *s_sw = reinterpret_cast<float *>(smem + FBL_OFF_SW) + 2 * w;
    float *s_comb = reinterpret_cast<float *>(smem + FBL_OFF_COMB);
    const uint32_t sx_at = smem_addr(s_sx + row), sw_at = smem_addr(s_sw + lane);
    pdl_wait();  // s_x comes from the previous kernel
    int ft = unit, fkb = 0, fn = 0;
    const float *fx = nullptr, *fw = nullptr;
    bool in0 = false, in1 = false, inw = false;
    auto fetch_tile = [&]() {
      int tm = 0, tn = 0;
      if (ft < ntiles) tiles.at(ft, tm, tn);
      const int m = tm * TM + m_cta + row;
      in0 = ft < ntiles && m < p.M;
      in1 = ft < ntiles && m + 32 < p.M;
      fx = p.sx + (in0 ? m : 0);
      inw = ft < ntiles && lane < 2;
      const int nb = GATE ? tn : min(2 * tn + lane, NB - 1);
      fw = (GATE && lane == 1 ? p.sw[1] : p.sw[0]) + (inw ? static_cast<size_t>(nb) * p.G : 0);
    };
    auto fetch = [&]() {
      const uint32_t slot = static_cast<uint32_t>(fn & (FBL_AHEAD - 1));
      const float *x = fx + static_cast<size_t>(kb0 + fkb) * p.M;
      if (in0 && DFK_IN_BOUNDS(kb0 + fkb < p.G, 32, p.err)) cp_async4(sx_at + slot * 512, x);
      if (in1) cp_async4(sx_at + slot * 512 + 128, x + 32);
      if (inw) cp_async4(sw_at + slot * 16, fw + kb0 + fkb);
      cp_async_commit();
      ++fn;
      if (++fkb == nkb) {
        fkb = 0;
        ft += nunits;
        fetch_tile();
      }
    };
    fetch_tile();
#pragma unroll 1
    for (int i = 0; i < FBL_AHEAD - 1; ++i) fetch();
#pragma unroll 1
    for (int it = 0; it < total; ++it) {
      const int slot = it & (FBL_AHEAD - 1), cs = it & (FBL_COMB - 1);
      cp_async_wait<FBL_AHEAD - 2>();
      __syncwarp();
      const float x0 = s_sx[slot * 128 + row], x1 = s_sx[slot * 128 + row + 32];
      const float w0 = s_sw[slot * 4], w1 = s_sw[slot * 4 + 1];
      fetch();  // into the slot of the group before this one
      // One barrier tells the epilogue that a half's sums and its scales are
      // there.  Group it - 2 is complete before `it` arrives on the same
      // barriers; its MMAs followed the epilogue's release of group it - 4, the
      // last to use this slot.
      uint64_t *full = &accfull[2 * (it & 1)];
      const uint32_t before = ((it >> 1) - 1) & 1;
      const bool ok = it < 2 || (fb_wait(&full[0], before, s_abort, p.err) &&
                                 fb_wait(&full[1], before, s_abort, p.err));
      if (!__all_sync(0xffffffffu, ok)) break;
      float *c = s_comb + cs * 256 + row;
      c[0] = x0 * w0;
      c[32] = x1 * w0;
      c[128] = x0 * w1;
      c[160] = x1 * w1;
      __syncwarp();
      if (lane < 2) mbar_arrive(&full[lane]);
    }
    cp_async_wait<0>();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(FBL_REGS_EPI));
    // ---- epilogue: thread = one token (TMEM lane) and half of the columns, 64 of
    // each CTA's weight rows (gated: 64 gate and the 64 matching up columns)
    const int ew = warp - 4, half = ew >> 2, q = warp & 3;
    const int row = 32 * q + lane;
    const uint32_t base = tmem + (static_cast<uint32_t>(32 * q) << 16);
    const float *s_comb = reinterpret_cast<const float *>(smem + FBL_OFF_COMB) + row;
    float *s_max = reinterpret_cast<float *>(smem + FBL_OFF_MAX);
    uint8_t *obuf = smem + FBL_OFF_OUT + ew * 2048;
    const uint32_t empty_at = cluster_map(smem_addr(&accempty[half]), lead);
    pdl_wait();  // the outputs may still be read by the previous kernel

    int it = 0, nth = 0;
    bool ok = true, rdy = false;
    for (int t = unit; ok && t < ntiles; t += nunits, ++nth) {
      uint64_t acc[64];  // pairs of neighbouring columns
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0ull;
      // One group at a time, 16 columns a step, the next 16 on their way; the
      // next group's barrier is tested in the shadow of the last sums.
      const uint32_t tb = base + 128 * half;
#pragma unroll 1
      for (int kb = 0; kb < nkb; ++kb) {
        const int ab = it & 1;
        if (!rdy) {
          ok = fb_wait(&accfull[2 * ab + half], (it >> 1) & 1, s_abort, p.err);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
        }
        tc_fence_after();
        uint32_t d[2][16];
        tmem_ld16(tb + ab * 256, d[0]);
        const float *sc = s_comb + (it & (FBL_COMB - 1)) * 256;
        const float s0 = sc[0], s1 = sc[128];
        ++it;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          tmem_wait16(d[c & 1]);
          if (c < 7) {
            tmem_ld16(tb + ab * 256 + 16 * (c + 1), d[(c + 1) & 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(empty_at + 16 * ab);
            rdy = __all_sync(0xffffffffu, mbar_test(&accfull[2 * (it & 1) + half], (it >> 1) & 1));
          }
          const uint64_t cc = c < 4 ? pack_f32x2(s0, s0) : pack_f32x2(s1, s1);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            acc[8 * c + e] = fma_f32x2(
                pack_f32x2(__uint_as_float(d[c & 1][2 * e]), __uint_as_float(d[c & 1][2 * e + 1])),
                cc, acc[8 * c + e]);
        }
      }
      if (!ok) break;
      if (!PAIR && ks > 1) {
        // ---- a share of a tile (each cluster has one): the partial sums go to
        // shared memory, token by token, once every MMA has read the ring
        ok = __all_sync(0xffffffffu, fb_wait(done, 0, s_abort, p.err));
        if (!ok) break;
        float *part = reinterpret_cast<float *>(smem + row * FBL_PART_ROW) + 64 * half;
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          float4 v;
          unpack_f32x2(acc[i], v.x, v.y);
          unpack_f32x2(acc[i + 1], v.z, v.w);
          *reinterpret_cast<float4 *>(part + (i < 32 ? 0 : 128) + 2 * (i & 31)) = v;
        }
        break;
      }
      // ---- the tile's output
      int tm, tn;
      tiles.at(t, tm, tn);
      const int m0 = tm * TM + m_cta + 32 * q;  // the warp's first row
      if constexpr (!GATE) {
        const int n0 = tn * 256 + 64 * half;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float lo, hi;
            unpack_f32x2(acc[16 * c + e], lo, hi);
            w[e] = pack_bf16x2(lo, hi);
          }
          fbl_stage(obuf, lane, w);
          fbl_store_bf16(p, obuf, lane, m0, n0 + (c & 1) * 32 + (c >> 1) * 128);
        }
      } else {
        const int n0 = tn * 128 + 64 * half;
        float h[64];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          float g0, g1, u0, u1;
          unpack_f32x2(acc[e], g0, g1);
          unpack_f32x2(acc[32 + e], u0, u1);
          h[2 * e] = fb_silu_mul(g0, u0);
          h[2 * e + 1] = fb_silu_mul(g1, u1);
        }
        if (p.y != nullptr) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(h[32 * c + 2 * e], h[32 * c + 2 * e + 1]);
            fbl_stage(obuf, lane, w);
            fbl_store_bf16(p, obuf, lane, m0, n0 + 32 * c);
          }
        } else {
          // the group's other 64 columns are in the warp with the same rows
          float mx = 0.f;
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (n0 + e < p.N) mx = max_nan(mx, fabsf(h[e]));
          // (two buffers: a warp that writes tile nth + 2 has seen the other
          // one at tile nth + 1, after its read of nth)
          float *mb = s_max + (nth & 1) * 256;
          mb[half * 128 + row] = mx;
          __syncwarp();
          if (lane == 0) mbar_arrive(&maxfull[q]);
          ok = __all_sync(0xffffffffu, fb_wait(&maxfull[q], nth & 1, s_abort, p.err));
          if (!ok) break;
          mx = max_nan(mx, mb[(1 - half) * 128 + row]);
          const FbScale f = fb_scale(mx);
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[e] = fb_codes4(h[4 * e], h[4 * e + 1], h[4 * e + 2], h[4 * e + 3], f);
          fbl_stage(obuf, lane, w);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 8 * i + (lane >> 2), c = lane & 3, m = m0 + r, col = n0 + 16 * c;
            const uint4 v = *reinterpret_cast<const uint4 *>(fbl_chunk(obuf, r, c));
            if (m < p.M && col < p.N && DFK_IN_BOUNDS(col + 16 <= p.N, 33, p.err))
              *reinterpret_cast<uint4 *>(p.qh + static_cast<size_t>(m) * p.N + col) = v;
          }
          __syncwarp();
          if (half == 0 && m0 + lane < p.M && DFK_IN_BOUNDS(tn < NB, 34, p.err))
            p.sh[static_cast<size_t>(tn) * p.M + m0 + lane] = f.s;
        }
      }
    }
  }

  // every wait above is bounded, so all CTAs of the cluster come here; the MMAs
  // have completed and the copies have landed before any leaves
  __syncthreads();
  if (tid == 0) {
    fb_wait(done, 0, nullptr, p.err);
    if (*s_abort) {
      const int issued = *s_issued;
      if (rank == lead)
        for (int i = max(0, issued - S); i < issued; ++i)
          fb_wait(&fullb[i % S], (i / S) & 1, nullptr, p.err);
      // copies that only one CTA of a pair issued are counted by no complete
      // phase: they land within microseconds, allow a millisecond
      const unsigned long long t0 = global_timer_ns();
      for (int i = 0; i < 100000 && global_timer_ns() - t0 < 1000000ull; ++i) __nanosleep(1000);
    }
  }
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) {
    if constexpr (PAIR) tmem_dealloc_pair(tmem, 512);
    else tmem_dealloc(tmem, 512);
  }
  if (!PAIR && ks > 1) {
    // ---- the cluster's shares added in rank order through distributed shared
    // memory: a token per warp and turn, spread over the CTAs
    if (warp >= 4 && !*s_abort) {
      int tm, tn;
      tiles.at(unit, tm, tn);
      const int nt = min(128, p.M - tm * 128);
      const int nv = GATE || tn * 256 + 128 < p.N ? 2 : 1;  // a second block of 128 columns
      for (int n = kr * 8 + (warp - 4); n < nt; n += 8 * ks) {
        float4 a[2];
        fb_sum_shares<2>(sbase + static_cast<uint32_t>(n * FBL_PART_ROW + 16 * lane), 512, ks, nv,
                         a);
        const int m = tm * 128 + n;
        if constexpr (GATE) {
          if (p.y == nullptr) fb_emit4_codes(p, m, tn, lane, a[0], a[1]);
          else fb_emit4<2>(p, m, tn, lane, a[0], a[1]);
        } else {
          fb_emit4<1>(p, m, 2 * tn, lane, a[0], a[0]);
          if (nv == 2) fb_emit4<1>(p, m, 2 * tn + 1, lane, a[1], a[1]);
        }
      }
    }
    cluster_sync_relaxed();  // no CTA leaves while its sums are being read
  }
}

const void *fb_large_kernel_fn(bool gate, bool pair) {
  return gate ? (pair ? reinterpret_cast<const void *>(&fb_large_kernel<true, true>)
                      : reinterpret_cast<const void *>(&fb_large_kernel<true, false>))
              : (pair ? reinterpret_cast<const void *>(&fb_large_kernel<false, true>)
                      : reinterpret_cast<const void *>(&fb_large_kernel<false, false>));
}

int fb_large_weight_box(bool pair) { return pair ? 128 : 64; }

cudaError_t launch_fb_large(bool gate, bool pair, int ks, const FbMaps &maps, const FbParams &p,
                            int sms, cudaStream_t st, bool pdl) {
  const int tokens = pair ? 256 : 128, cluster = pair ? 2 : ks;
  const long long tm = (p.M + tokens - 1) / tokens;
  const long long tn = gate ? (p.N + 127) / 128 : (p.N + 255) / 256;
  const long long units = ks > 1 ? tm * tn : std::min<long long>(sms / cluster, tm * tn);
  FbMaps mp = maps;
  FbParams pp = p;
  const long long tile_bytes = static_cast<long long>(tokens) * p.G * FB_GROUP;
  pp.band = static_cast<int>(std::min(64LL, std::max(4LL, FBL_BAND_BYTES / tile_bytes)));
  void *args[] = {&mp, &pp};
  return launch_kernel(fb_large_kernel_fn(gate, pair), dim3(static_cast<unsigned>(cluster * units)),
                       dim3(FBL_THREADS), FBL_SMEM, st, pdl, args,
                       static_cast<unsigned>(cluster));
}

}  // namespace dfk

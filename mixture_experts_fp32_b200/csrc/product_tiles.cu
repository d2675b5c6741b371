// out = A W^T with e4m3 operands and fp32 block scales, more rows than weight_stream.cuh takes:
//
//   out[m, n] = sum_kb sa[m, kb] * sw[n / 128, kb] * sum_{k in kb} a[m, k] * w[n, k]
//
// The scale changes every 128 K, and arbitrary fp32 scales cannot be given to the tensor
// core's block-scaled kinds (they take powers of two), so each block of 128 K is multiplied
// into tensor-memory buffers of its own (exact products, fp32 sums), and the epilogue warps
// add them to fp32 registers with its scale.  That is what bounds the kernel: a block's
// MMAs take 512 clocks, its FMAs 290, and its way through tensor memory more than either (about
// 900 clocks from an MMA's issue until its completion is seen, 500 until the buffer has been
// read and returned).  So the two warpgroups of the epilogue have a half of the features each
// and two buffers of their own for it: while one waits for its half or reads it, the other
// adds.  (One pair of buffers for both: 880 clocks a block.)
//
// A tile is 256 rows x 256 features, by the two CTAs of a cluster with cta_group::2 MMAs: each
// stages its own 128 rows of A and one half (128 rows) of the weights, 32 KB of shared
// memory a block where a one-CTA 128 x 256 tile stages 48, and receives its 128 rows x 256
// columns in its own tensor memory.  The even CTA issues the MMAs and owns the stage barriers; the
// odd CTA's loads complete there, and its epilogue warps return buffers by remote arrivals.
// No load is multicast.
//
// A stage is two K blocks, which one TMA instruction brings for A and one for W (a 3-D map of
// 128-byte columns; where K is no multiple of 128 the last column has no 128 bytes, and two
// 2-D loads take the place of each).
//
// Warpgroup 0: TMA producer, MMA issuer; warpgroups 1 and 2 (8 warps) promote and finish,
// with the registers warpgroup 0 gives back: a thread has one row (its tensor-memory lane)
// and 128 columns.
//
// Fewer tiles than cluster pairs: K is cut into `splits` parts of a tile.  Each stores its sums
// and, when all have arrived, finishes its part of the columns, adding the parts in order, so
// results do not depend on timing.  (The last part to arrive finishing all: 256 x 4096 x 7168
// 31 us.)
#include <cudaTypedefs.h>

#include <atomic>

#include "product.cuh"

namespace moe {
namespace {

constexpr int BM = 128;                        // rows of A per CTA
constexpr int BN = 256;                        // features per tile; half of them staged per CTA
constexpr int BH = BN / 2;                     // features of a half: 64 of them staged per CTA
constexpr int BK = 128;                        // e4m3 values (bytes) per K block
constexpr int kEpiWarps = 8;
constexpr int kThreads = 384;
// 12 warps leave each SM sub-partition three: 168 registers a thread at launch.  Warpgroup 0
// drops to 24, warpgroups 1 and 2 rise to 240: 128 * 24 + 256 * 240 = 384 * 168.
constexpr int kLaunchRegs = 168;
constexpr int kProducerRegs = 24;
constexpr int kEpilogueRegs = 240;
static_assert(128 * kProducerRegs + 256 * kEpilogueRegs == kThreads * kLaunchRegs,
              "register shares must add up to the launch's registers");
constexpr int A_BYTES = BM * BK;
constexpr int B_BYTES = (BN / 2) * BK;
constexpr int STAGES = 3;                      // of two K blocks
constexpr int STG_BYTES = 8 * 256;             // a warp's staged output: 8 rows x 256 bytes
constexpr unsigned long long kTeardownNs = 100000000ull;

struct TileSmem {
  alignas(1024) uint8_t a[STAGES][2 * A_BYTES];
  alignas(1024) uint8_t b[STAGES][2 * B_BYTES];   // [half][K block][64 rows]
  alignas(16) uint8_t stg[kEpiWarps][STG_BYTES];
  uint64_t full[STAGES];                       // even CTA: stage loaded in both CTAs
  uint64_t empty[STAGES];                      // stage consumed by the pair's MMAs
  uint64_t pfull[2][2];                        // [half][buffer] written (both CTAs)
  uint64_t pempty[2][2];                        // even CTA: buffer read by its 8 epilogue warps
  uint64_t teardown;
  uint32_t tmem;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Address of the same shared-memory object in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_to_rank(uint32_t smem_addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr), "r"(rank));
  return r;
}
// Remote arrival that publishes no memory: it returns a tensor-memory buffer, whose reads
// tcgen05.wait::ld has completed and tcgen05.fence::before_thread_sync has ordered before.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
               "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 2-D tiled TMA load (no multicast) into this CTA's shared memory whose bytes complete on an
// mbarrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* m, int x, int y,
                                              uint32_t bar_cluster, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar_cluster), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_pair_3d(uint32_t dst, const CUtensorMap* m, int x, int y,
                                                 int z, uint32_t bar_cluster, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar_cluster), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_pair_4d(uint32_t dst, const CUtensorMap* m, int x, int y,
                                                 int z, int w, uint32_t bar_cluster,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar_cluster),
      "l"(policy)
      : "memory");
}
// D[tmem of both CTAs] (+)= A[smem of both] * B[smem of both]^T, M = 256, N = 128.
__device__ __forceinline__ void umma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t accumulate) {
  constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(BH >> 3) << 17) |
                             ((uint32_t)(2 * BM >> 4) << 24);
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on the mbarrier at this offset in both CTAs once the pair MMAs issued so far are done.
__device__ __forceinline__ void umma_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(bar), "h"((uint16_t)0x3)
      : "memory");
}

struct TileArgs {
  ProductArgs p;
  int tiles_m, splits, kb_per_split, total;    // total = tiles * splits items; kb_per_split even
  bool columns;                                // maps of 128-byte columns (K a multiple of 128)
};

struct Item {
  int tile, split, m0, n0, kb0, kb1;
};
__device__ __forceinline__ Item item_of(int i, const TileArgs& t) {
  Item o;
  o.tile = i / t.splits;
  o.split = i - o.tile * t.splits;
  const int f = o.tile / t.tiles_m;            // feature tile outer, row tile inner
  o.n0 = f * BN;
  o.m0 = (o.tile - f * t.tiles_m) * 2 * BM;
  o.kb0 = o.split * t.kb_per_split;
  o.kb1 = min(t.p.kb, o.kb0 + t.kb_per_split);
  return o;
}

// A warp's 32 rows (m0 ..) x 128 columns (n0 ..) out, 256 bytes of a row at a time: the lanes of
// 8 rows put their segments into shared memory (16-byte chunk c of row j at slot c ^ j: no bank
// conflicts either way), then every store instruction covers two whole segments, lanes 0 - 15
// one row, 16 - 31 the next.  `get(c)`: columns 2c, 2c + 1 of this lane's row.
template <typename OT, class G>
__device__ __forceinline__ void store_rows(const ProductArgs& p, uint8_t* stg, int m0, int n0,
                                           G&& get) {
  const int lane = threadIdx.x & 31;
  constexpr int kVals = 256 / sizeof(OT);      // columns of a segment
  constexpr int kChunk = 16 / sizeof(OT);      // and of a 16-byte chunk
  const uint32_t s = smem_u32(stg);
  OT* out = static_cast<OT*>(p.out);
  const bool vec = (reinterpret_cast<uintptr_t>(out) & 15u) == 0 && (p.ldo * sizeof(OT)) % 16 == 0;
#pragma unroll
  for (int c0 = 0; c0 < 128; c0 += kVals) {
    uint32_t pk[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) {
      if (sizeof(OT) == 2) {
        const float2 v = get(i);
        const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
        pk[i] = *reinterpret_cast<const uint32_t*>(&b);
      } else {
        const float2 v = get((c0 + i) / 2);
        pk[i] = __float_as_uint((i & 1) ? v.y : v.x);
      }
    }
#pragma unroll 1
    for (int rnd = 0; rnd < 4; ++rnd) {
      if (m0 + 8 * rnd >= p.M) break;
      if ((lane >> 3) == rnd) {
        const int j = lane & 7;
#pragma unroll
        for (int w = 0; w < 16; ++w)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(s + j * 256 +
                                                                        ((w ^ j) & 15) * 16),
                       "r"(pk[4 * w]), "r"(pk[4 * w + 1]), "r"(pk[4 * w + 2]), "r"(pk[4 * w + 3])
                       : "memory");
      }
      __syncwarp();
      if (vec) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = 2 * i + (lane >> 4), c = lane & 15;
          uint4 o;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(o.x), "=r"(o.y), "=r"(o.z), "=r"(o.w)
                       : "r"(s + j * 256 + ((c ^ j) & 15) * 16)
                       : "memory");
          const int m = m0 + rnd * 8 + j, n = n0 + c0 + c * kChunk;
          if (m < p.M && n < p.N) {
            OT* dst = out + m * p.ldo + n;
            if (n + kChunk <= p.N) {
              *reinterpret_cast<uint4*>(dst) = o;
            } else {
              const OT* v = reinterpret_cast<const OT*>(&o);
#pragma unroll
              for (int e = 0; e < kChunk; ++e)
                if (n + e < p.N) dst[e] = v[e];
            }
          }
        }
      } else {
        // rows that begin anywhere: consecutive lanes store consecutive values
        OT v[8][kVals / 32];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int i = 0; i < kVals / 32; ++i) {
            const int e = lane + 32 * i;
            v[j][i] = *reinterpret_cast<const OT*>(stg + j * 256 + ((e / kChunk ^ j) & 15) * 16 +
                                                   e % kChunk * sizeof(OT));
          }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int m = m0 + rnd * 8 + j;
#pragma unroll
          for (int i = 0; i < kVals / 32; ++i) {
            const int n = n0 + c0 + lane + 32 * i;
            if (m < p.M && n < p.N) out[m * p.ldo + n] = v[j][i];
          }
        }
      }
      __syncwarp();
    }
  }
}

template <bool F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    product_tiles_kernel(const __grid_constant__ CUtensorMap tmA,
                         const __grid_constant__ CUtensorMap tmW, const TileArgs t) {
  extern __shared__ uint8_t smem_raw[];
  TileSmem& s = *reinterpret_cast<TileSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const ProductArgs& p = t.p;
  constexpr unsigned int kBit = MOE_DEV_WAIT_TIMEOUT_PRODUCT;
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();          // 0: issues the MMAs
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&s.pfull[i >> 1][i & 1]), 1);
      mbar_init(smem_u32(&s.pempty[i >> 1][i & 1]), kEpiWarps);   // four of either CTA
    }
    mbar_init(smem_u32(&s.teardown), 1);
    fence_mbarrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmW);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&s.tmem)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();        // the peer's barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s.tmem, 0);

  if (warp < 4) {
    regs_dec<kProducerRegs>();
    if (warp == 0) {
      // ------------------------------------------------------------ TMA producer
      const uint64_t pol = policy_evict_normal();
      int stage = 0;
      uint32_t phase = 0, issued = 0, parity = 0;
      bool ok = true;
      const uint32_t full0 = map_to_rank(smem_u32(&s.full[0]), 0);   // the even CTA's barriers
      for (int i = pair; i < t.total && ok; i += npairs) {
        const Item it = item_of(i, t);
        const int arow = it.m0 + BM * (int)rank, wrow = it.n0 + (BH / 2) * (int)rank;
        for (int kb = it.kb0; kb < it.kb1; kb += 2) {
          ok = ws_wait(smem_u32(&s.empty[stage]), phase ^ 1u, p.wait_limit_ns,
                                      p.status, kBit);
          if (!ok) break;
          const uint32_t own = smem_u32(&s.full[stage]);
          const uint32_t fb = full0 + stage * (uint32_t)sizeof(uint64_t);
          const uint32_t a = smem_u32(s.a[stage]), b = smem_u32(s.b[stage]);
          if (elect_one()) {
            if (rank == 0) mbar_arrive_expect_tx(own, 4 * (A_BYTES + B_BYTES));
            if (t.columns) {
              tma_load_pair_4d(a, &tmA, 0, arow, kb, 0, fb, pol);
              tma_load_pair_3d(b, &tmW, 0, wrow, kb, fb, pol);
              tma_load_pair_3d(b + B_BYTES, &tmW, 0, wrow + BH, kb, fb, pol);
            } else {
#pragma unroll
              for (int j = 0; j < 2; ++j) {           // past the end of K: zeros
                tma_load_pair_3d(a + j * A_BYTES, &tmA, (kb + j) * BK, arow, 0, fb, pol);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  tma_load_pair(b + h * B_BYTES + j * (B_BYTES / 2), &tmW, (kb + j) * BK,
                                wrow + h * BH, fb, pol);
              }
            }
          }
          __syncwarp();
          issued |= 1u << stage;
          parity = (parity & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      // no load may still be writing when the CTA leaves: wait until the MMAs have consumed the
      // last load of every stage (which follows its arrival)
      for (int i = 0; i < STAGES; ++i)
        if ((issued >> i) & 1u)
          mbar_wait_sleep_warp(smem_u32(&s.empty[i]), (parity >> i) & 1u, kTeardownNs, p.status,
                               kBit);
    } else if (warp == 1 && rank == 0) {
      // -------------------------------------------------------------- MMA issuer
      int stage = 0;
      uint32_t phase = 0, count = 0;
      bool ok = true, any = false;
      for (int i = pair; i < t.total && ok; i += npairs) {
        const Item it = item_of(i, t);
        for (int kb = it.kb0; kb < it.kb1 && ok; kb += 2) {
          ok = ws_wait(smem_u32(&s.full[stage]), phase, p.wait_limit_ns, p.status,
                                      kBit);
          if (!ok) break;
          const uint64_t a = smem_desc_sw128(smem_u32(s.a[stage]));
          const uint64_t b = smem_desc_sw128(smem_u32(s.b[stage]));
          const int blocks = min(2, it.kb1 - kb);
          for (int j = 0; j < blocks && ok; ++j, ++count) {
            const uint32_t pb = count & 1u, use = count >> 1;
            const uint64_t aj = a + j * (A_BYTES >> 4);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              ok = ok && ws_wait(smem_u32(&s.pempty[h][pb]), (use & 1u) ^ 1u, p.wait_limit_ns,
                                 p.status, kBit);
              if (!ok) break;
              tc_fence_after();
              const uint64_t bj = b + (h * B_BYTES + j * (B_BYTES / 2) >> 4);
              const uint32_t dst = tmem + (2 * h + pb) * BH, full = smem_u32(&s.pfull[h][pb]);
              const uint32_t empty = smem_u32(&s.empty[stage]);
              if (elect_one()) {
#pragma unroll
                for (int k = 0; k < BK / 32; ++k)   // +32 bytes per K step = 2 in the address field
                  umma_pair(dst, aj + 2 * k, bj + 2 * k, k != 0);
                umma_commit_pair(full);
                if (h == 1 && j + 1 == blocks) umma_commit_pair(empty);
              }
              __syncwarp();
              any = true;
            }
          }
          if (!ok) break;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (any) {
        if (elect_one()) umma_commit_pair(smem_u32(&s.teardown));
        __syncwarp();
        mbar_wait_sleep_warp(smem_u32(&s.teardown), 0, kTeardownNs, p.status, kBit);
      }
    }
    __syncwarp();
  } else {
    regs_inc<kEpilogueRegs>();
    // ---------------------------------------------------- promotion and epilogue
    // After an expired wait the warps keep walking without further waits, so that every named
    // barrier is reached.
    const int q = warp & 3, hh = (warp - 4) >> 2;   // tensor-memory lanes, column half
    const uint32_t pempty0 = map_to_rank(smem_u32(&s.pempty[hh][0]), 0);
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + hh * 2 * BH;
    uint32_t count = 0;
    bool ok = true;
    // scales two blocks ahead, one set for even and one for odd blocks; an item's first ones are
    // asked for before the item before it is stored
    float xa[2], xw[2];
    const float *sa, *sw;
    auto first_scales = [&](const Item& it) {
      // rows and columns past the end read the last ones' scales (in bounds, not used)
      sa = p.sa + (size_t)min(it.m0 + BM * (int)rank + q * 32 + lane, p.M - 1) * p.kb;
      sw = p.sw + (size_t)(min(it.n0 + hh * BH, p.N - 1) / 128) * p.kb;
      const int next = min(it.kb0 + 1, it.kb1 - 1);
      xa[0] = ldg_ahead(sa + it.kb0);
      xw[0] = ldg_ahead(sw + it.kb0);
      xa[1] = ldg_ahead(sa + next);
      xw[1] = ldg_ahead(sw + next);
    };
    if (pair < t.total) first_scales(item_of(pair, t));
    for (int i = pair; i < t.total; i += npairs) {
      const Item it = item_of(i, t);
      const int m0 = it.m0 + BM * (int)rank + q * 32, n0 = it.n0 + hh * BH;
      const bool warp_live = m0 < p.M && n0 < p.N;
      float2 acc[64];
#pragma unroll
      for (int c = 0; c < 64; ++c) acc[c] = make_float2(0.f, 0.f);
      for (int kk = it.kb0; kk < it.kb1; kk += 2) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int kb = kk + j;
          if (kb >= it.kb1) break;
          const float f = xa[j] * xw[j];
          const float2 f2 = make_float2(f, f);
          if (kb + 2 < it.kb1) {
            xa[j] = ldg_ahead(sa + kb + 2);
            xw[j] = ldg_ahead(sw + kb + 2);
          }
          const uint32_t pb = count & 1u, use = count >> 1;
          ++count;
          if (ok) ok = ws_wait(smem_u32(&s.pfull[hh][pb]), use & 1u, p.wait_limit_ns, p.status, kBit);
          if (!ok) continue;
          tc_fence_after();
          const uint32_t at = lanes + pb * BH;
          uint32_t ra[32], rb[32];
          if (warp_live) {
            // half the columns at a time, and the buffer goes back before the last 64 are added:
            // what an MMA waits for is the buffer
            tmem_ld_2x16(at, at + 16, ra);
            tmem_ld_2x16(at + 32, at + 48, rb);
            tmem_ld_wait_tied2(ra, rb);
            promote16(acc, 0, ra, f2);
            tmem_ld_2x16(at + 64, at + 80, ra);
            promote16(acc, 16, rb, f2);
            tmem_ld_2x16(at + 96, at + 112, rb);
            tmem_ld_wait_tied2(ra, rb);
          }
          tc_fence_before();
          __syncwarp();
          if (rank == 0) {
            if (elect_one()) mbar_arrive(smem_u32(&s.pempty[hh][pb]));
          } else if (elect_one()) {
            mbar_arrive_remote(pempty0 + pb * (uint32_t)sizeof(uint64_t));
          }
          if (warp_live) {
            promote16(acc, 32, ra, f2);
            promote16(acc, 48, rb, f2);
          }
        }
      }
      if (i + npairs < t.total) first_scales(item_of(i + npairs, t));
      if (t.splits > 1) {
        // this CTA's partial sums of a part of the tile: [column / 4][thread][4]
        auto part_of = [&](int sp) {
          return reinterpret_cast<float4*>(p.part) +
                 ((size_t)(it.tile * t.splits + sp) * 2 + rank) * (32 * 256) + threadIdx.x - 128;
        };
        if (warp_live) {
          float4* o = part_of(it.split);
#pragma unroll
          for (int c = 0; c < 32; ++c)
            __stcg(o + c * 256,
                   make_float4(acc[2 * c].x, acc[2 * c].y, acc[2 * c + 1].x, acc[2 * c + 1].y));
        }
        named_bar_sync(1, kEpiWarps * 32);
        unsigned int* counter = p.counters + it.tile * 2 + rank;
        if (warp == 4 && elect_one())
          asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(counter) : "memory");
        if (warp_live && ok) {
          const uint64_t t0 = global_timer_ns();
          while (__any_sync(0xffffffffu, ld_acquire_gpu(counter) < (unsigned int)t.splits)) {
            if (__any_sync(0xffffffffu, global_timer_ns() - t0 >= p.wait_limit_ns)) {
              if (lane == 0) atomicOr(p.status, kBit);
              ok = false;
              break;
            }
          }
          const int c1 = ok ? 32 * (it.split + 1) / t.splits : 0;
#pragma unroll 1
          for (int c0 = 32 * it.split / t.splits; c0 < c1; c0 += 8) {
            float4 sum[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) sum[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (int sp = 0; sp < t.splits; sp += 4) {
              float4 v[4][8];                         // all on their way at once
#pragma unroll
              for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int c = 0; c < 8; ++c)
                  v[j][c] = sp + j < t.splits && c0 + c < c1
                                ? __ldcg(part_of(sp + j) + (c0 + c) * 256)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
              for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                  sum[c].x += v[j][c].x;
                  sum[c].y += v[j][c].y;
                  sum[c].z += v[j][c].z;
                  sum[c].w += v[j][c].w;
                }
            }
#pragma unroll
            for (int c = 0; c < 8; ++c)
              if (m0 + lane < p.M && c0 + c < c1)
                store_out4(p, m0 + lane, n0 + 4 * (c0 + c), sum[c]);
          }
        }
      } else if (ok && warp_live) {
        auto get = [&](int c) { return acc[c]; };
        if (F32)
          store_rows<float>(p, s.stg[warp - 4], m0, n0, get);
        else
          store_rows<__nv_bfloat16>(p, s.stg[warp - 4], m0, n0, get);
      }
    }
  }

  // Neither CTA leaves (or frees tensor memory) while the other may still arrive on its
  // barriers or have the tensor core read its shared memory.
  tc_fence_before();
  __syncthreads();
  // odd CTA: the pair's last commit arrives here too.  Not waited for before its roles have
  // finished: a limit that ran from the launch on would bound the whole product.
  if (warp == 1 && rank != 0 && pair < t.total)
    mbar_wait_sleep_warp(smem_u32(&s.teardown), 0, kTeardownNs, p.status, kBit);
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

std::atomic<int> resident_pairs{kProductPairs};       // clusters a device holds at once, at most

// The register shares of the warpgroups only add up if the kernel was built with exactly
// kLaunchRegs registers a thread; anything else is refused rather than launched (a
// mismatched split would wait forever).
template <bool F32>
cudaError_t prepare() {
  static_assert(sizeof(TileSmem) + 1024 <= 227 * 1024, "shared memory of one CTA");
  cudaFuncAttributes attr;
  cudaError_t e = cudaFuncGetAttributes(&attr, product_tiles_kernel<F32>);
  if (e != cudaSuccess) return e;
  if (attr.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(product_tiles_kernel<F32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)sizeof(TileSmem) + 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * kProductPairs, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = sizeof(TileSmem) + 1024;
  int pairs = 0;
  e = cudaOccupancyMaxActiveClusters(&pairs, product_tiles_kernel<F32>, &cfg);
  if (e != cudaSuccess) return e;
  if (pairs < 1) return cudaErrorInvalidConfiguration;
  if (pairs < resident_pairs.load()) resident_pairs = pairs;
  return cudaSuccess;
}

// Maps of a tensor of less than 128 KB load these boxes at a fraction of the rate: 40 x 18944 x 2048
// took 39 us with A's 80 KB mapped as they are, 64 rows (128 KB) 18.5.  So A's maps get one more
// dimension, of as many copies as 128 KB take, of which only the first is ever addressed (now
// 18.5 us).  The weight stream's smaller boxes load as well either way.
uint64_t copies(uint64_t bytes) { return ((1 << 17) + bytes - 1) / bytes; }
// Row-major bytes [rows, K], in boxes of 128 columns of `box_rows` rows.
bool row_map(CUtensorMap* m, const void* a, uint64_t K, uint64_t rows, int box_rows) {
  const uint64_t dims[3] = {K, rows, copies(K * rows)}, strides[2] = {K, K * rows};
  const uint32_t box[3] = {BK, (uint32_t)box_rows, 1};
  return ws_map_nd(m, a, 3, dims, strides, box);
}
// The same as [K / 128][rows][128], in boxes of two columns; rank 4: with copies.
bool column_map(CUtensorMap* m, const void* w, uint64_t K, uint64_t rows, int box_rows, int rank) {
  const uint64_t dims[4] = {BK, rows, K / BK, copies(K * rows)}, strides[3] = {K, BK, K * rows};
  const uint32_t box[4] = {BK, (uint32_t)box_rows, 2, 1};
  return ws_map_nd(m, w, rank, dims, strides, box);
}

// How the tiles are cut: K of each in `splits` parts where there are fewer tiles than pairs.  A block
// of K takes 800 clocks, joining n parts 10000 (the partial sums' way) and 20000 / n (the
// finishing) and 500 n (16 tiles of 56 blocks: 22.6 us in four parts, 33 whole; 37 tiles of 28
// blocks: 27 us in halves, 21 whole).
struct TilePlan {
  long long tiles, clocks;
  int tiles_m, pairs, splits;
  TilePlan(const ProductArgs& p, int num_sms) {
    tiles_m = (p.M + 2 * BM - 1) / (2 * BM);
    tiles = (long long)tiles_m * ((p.N + BN - 1) / BN);
    const int most = resident_pairs.load();
    pairs = num_sms / 2 < most ? num_sms / 2 : most;
    const auto cost = [&](int n) {
      return (p.kb + n - 1) / n * 800ll + (n > 1 ? 10000 + 20000 / n + 500 * n : 0);
    };
    splits = 1;
    if (tiles < pairs)
      for (int n = 2; n * tiles <= pairs && n <= p.kb; ++n)
        if (cost(n) < cost(splits)) splits = n;
    clocks = (tiles + pairs - 1) / pairs * cost(splits);
  }
};

}  // namespace

cudaError_t prepare_product_tiles() {
  const cudaError_t e = prepare<false>();
  return e == cudaSuccess ? prepare<true>() : e;
}

long long product_tiles_clocks(const ProductArgs& p, int num_sms) {
  return TilePlan(p, num_sms).clocks;
}

cudaError_t launch_product_tiles(const ProductArgs& p, int num_sms, cudaStream_t st) {
  TileArgs t;
  t.columns = p.K % BK == 0;
  CUtensorMap ma, mw;
  if (t.columns
          ? !column_map(&ma, p.a, p.K, p.M, BM, 4) || !column_map(&mw, p.w, p.K, p.N, BH / 2, 3)
          : !row_map(&ma, p.a, p.K, p.M, BM) || !ws_map(&mw, p.w, p.K, p.N, BH / 2))
    return cudaErrorInvalidValue;
  const TilePlan plan(p, num_sms);
  if (plan.tiles > (1 << 29)) return cudaErrorInvalidValue;
  const int pairs = plan.pairs, splits = plan.splits;
  t.p = p;
  t.tiles_m = plan.tiles_m;
  t.kb_per_split = (p.kb + splits - 1) / splits;
  t.kb_per_split += t.kb_per_split & 1;
  t.splits = (p.kb + t.kb_per_split - 1) / t.kb_per_split;
  t.total = (int)plan.tiles * t.splits;
  const int grid = 2 * (t.total < pairs ? t.total : pairs);
  const cudaError_t e = cudaMemsetAsync(p.status, 0, product_head_bytes(p), st);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = sizeof(TileSmem) + 1024;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];                        // the parts of a tile wait for one another
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = t.splits > 1 ? 1 : 0;
  return p.f32 ? cudaLaunchKernelEx(&cfg, product_tiles_kernel<true>, ma, mw, t)
               : cudaLaunchKernelEx(&cfg, product_tiles_kernel<false>, ma, mw, t);
}

}  // namespace moe

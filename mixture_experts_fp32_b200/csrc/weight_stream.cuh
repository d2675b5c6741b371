// Streaming a weight matrix past a few activation rows: the pieces shared by the
// few-token layer and the block-scaled product of few rows.
//
// Every weight comes from HBM once and meets 32 activation rows at most, so both are bound by
// HBM, not by arithmetic: at 6.5 TB/s an SM receives about 23 bytes of weights a clock, 256
// rows x 128 bytes of K every 1400 clocks.  (A product of 33 to 128 rows is two to four blocks of
// 32 of them: these bring the weights to shared memory once each, after the first from L2, and
// share its rate.)  What matters is that nothing else takes longer than that, and that loads
// never pause:
//  - weights travel by TMA into a ring of stages in shared memory (256 weight rows x 128
//    bytes of K, two boxes of 128 rows), 160 KB or more a CTA in flight, by a producer that
//    runs on across tiles, barriers and phases;
//  - tcgen05 multiplies straight from shared memory, so that no instruction handles a
//    single weight, with the weights on the N side (256) and the few activation rows on the
//    M side (128, of which the rest is whatever lies behind them in shared memory: rows of
//    a product do not meet).  Four MMAs of 128 x 256 take 512 clocks, so a stage's weights
//    pass at 64 bytes a clock, and a finished row lies in one tensor-memory lane, which
//    few promoters reach; weights on the M side would need 360 clocks and four times the
//    promoters' loads, and neither is what bounds it.
//    The same product with warp-wide mma.sync took 330 instructions a warp and stage;
//  - a second producer brings the activation rows, so that weights can be under way before
//    the activations they will meet have been computed;
//  - what a launch runs once waits for its instructions longer than it runs, and beside full
//    rings every trip to L2 takes up to 4 us: the code between the phases is short loops and
//    its loads go out together;
//  - block scales change every 128 bytes of K (FP8): each stage is multiplied into one of
//    two tensor-memory buffers, and four promoter warps (the ones that can read the first
//    32 lanes, 64 columns each) add it to their fp32 sums with its scale.  Otherwise a
//    buffer takes a whole run of K.
//
// Work is cut into units of one stage.  Each CTA takes a contiguous range of the units
// (within one unit of an even split, whatever the shapes).  A tile whose units fall to
// several CTAs meets in global memory: each stores its partial sums where zeros lay, and
// who finishes a part of the tile reads them until none is zero, so a value announces
// itself (a sum of +0 travels as -0, which adds the same).  No counter, no fence, no order of
// arrival: one trip to L2.  (Counters with the last to arrive finishing took 8000 clocks
// and more beside a full ring of loads.)  The CTAs in whose range the tile comes last share
// the finishing; the last of its CTAs, which has it first, has long gone on by then.  Sums
// are added in a fixed order, so results do not depend on timing.  The CTAs wait for one
// another: cooperative launches.
//
// Fifteen warps: 1 weight producer, 2 MMA issuer, 3 activation producer; promoters 0, 4, 8, 12
// (lane: activation row; warp / 4: columns, i.e. weight rows, 64 (warp / 4) .. + 63); the
// other eight are workers, who take a finished tile from shared memory while the promoters
// are at the next one.
#pragma once

#include "moe_internal.cuh"

namespace moe {

constexpr int kWsRows = 256;                  // weight rows of a tile
constexpr int kWsBytes = 128;                 // bytes of K of a stage
constexpr int kWsBoxRows = 128;               // rows of a TMA box of weights
constexpr int kWsStageBytes = kWsRows * kWsBytes;
constexpr int kWsWorkers = 8;                 // warps
constexpr int kWsThreads = kWsWorkers * 32;   // worker threads
constexpr int kWsBlock = 15 * 32;
constexpr int kWsCols = kWsRows / 4;          // columns of a promoter
constexpr int kWsTilePitch = kWsRows + 4;     // a finished tile in shared memory: rows apart
constexpr unsigned long long kWsDrainNs = 1000000000ull;
// FP8: scales of a stage (of its activation rows, and of its two blocks of 128 weight rows)
// lie in a ring of slots.  No barrier guards a slot: the activation producer reaches stage
// u + kWsSlots only after the MMAs of stage u + kWsSlots - STAGES, which waited for the
// promoters to read the buffer two stages before that.
constexpr int kWsSlots = 16;

// Shared memory of the stream.  ROWS: activation rows brought (16 or 32), TILE: rows of a
// finished tile.
template <bool FP8_, int ROWS_, int TILE, int STAGES_>
struct WsSmem {
  static constexpr bool FP8 = FP8_;
  static constexpr int ROWS = ROWS_, STAGES = STAGES_;
  static_assert(STAGES + 2 < kWsSlots, "slots of scales");
  alignas(1024) uint8_t x[STAGES][ROWS * kWsBytes];   // MMAs read 128 rows from here: into w
  alignas(1024) uint8_t w[STAGES][kWsStageBytes];
  alignas(16) float tile[TILE][kWsTilePitch];
  float scale[kWsSlots][ROWS + 2];
  uint64_t full_w[STAGES], full_x[STAGES], empty[STAGES], dfull[2], dempty[2], teardown;
  uint32_t tmem;
};

// Tensor map of a row-major matrix [rows, row_bytes] in boxes of box_rows x 128 bytes with
// the 128-byte swizzle; what lies past its end reads as zero.
bool ws_map(CUtensorMap* m, const void* w, uint64_t row_bytes, uint64_t rows, int box_rows);
// Any tensor of bytes: `rank` extents, the strides of all but the first, and the box.
bool ws_map_nd(CUtensorMap* m, const void* w, int rank, const uint64_t* dims,
               const uint64_t* strides, const uint32_t* box);

#if defined(__CUDACC__)

// The split of `tiles` tiles of `per` units over the CTAs: contiguous ranges, the first `more`
// CTAs one unit more than `each`, the CTAs behind the last unit none.  Even over all CTAs,
// unless that leaves one fewer than kWsLeast units: sharing a tile costs its CTAs a trip
// through L2, 2000 clocks or more where a unit takes 800 to 1400, so small work goes to fewer
// CTAs, whole tiles where these are short.
constexpr int kWsLeast = 3;
struct WsSplit {
  int each, more;
  __host__ __device__ __forceinline__ WsSplit(int tiles, int per, int ctas) {
    const int units = tiles * per;
    if (units < ctas * kWsLeast)
      ctas = tiles < ctas && per <= 2 * kWsLeast ? tiles
                                                 : units / kWsLeast > 0 ? units / kWsLeast : 1;
    each = ctas > 0 ? units / ctas : 0;
    more = units - each * ctas;
    last = ctas;
  }
  int last;                                   // CTAs that take part
  // no tile has several CTAs
  __host__ __device__ __forceinline__ bool whole(int per) const {
    return each % per == 0 && more == 0;
  }
  __device__ __forceinline__ int begin(int cta) const {
    const int b = min(cta, last);
    return b * each + min(b, more);
  }
  __device__ __forceinline__ int owner(int u) const {
    const int head = more * (each + 1);
    return u < head ? u / (each + 1) : more + (u - head) / each;
  }
};


// The sharers of the tile that begins at unit t0: CTAs b0 .. b1.
struct WsShare {
  int b0, b1;
  __device__ __forceinline__ WsShare(const WsSplit& split, int t0, int per)
      : b0(split.owner(t0)), b1(split.owner(t0 + per - 1)) {}
  __device__ __forceinline__ int finishers() const { return max(b1 - b0, 1); }
};
// CTA b's partial tile [rows][kWsRows]: of the tile that its range begins inside of, or (tail)
// of the one that its range is first to touch.  part: [head, tail][kWsCtas].
__device__ __forceinline__ float* ws_partial(float* part, int rows, int b, bool tail) {
  return part + (size_t)((tail ? kWsCtas : 0) + b) * rows * kWsRows;
}

// One lane of a warp in step, chosen by the hardware.  Instructions of the tensor core and the
// TMA take their operands from registers that a warp's lanes share; issued under this vote, in
// code that the whole warp runs, they find them there.  Under a comparison of the thread's
// index every operand is carried over first: 100 clocks an instruction, so that four MMAs and
// their commits (512 clocks of work) took 880.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.b32 %0, 1, 0, P;\n\t}"
      : "=r"(p));
  return p != 0;
}
// The warp's index, as a value that its lanes share.
__device__ __forceinline__ int warp_index() {
  return __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
}

// Bounded wait taken by a whole warp (warp-uniform result): a limit of 0 gives up at once
// unless the phase is already complete, any other suspends between looks.
__device__ __forceinline__ bool ws_wait(uint32_t bar, uint32_t parity, unsigned long long limit_ns,
                                        unsigned int* status, unsigned int bit) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  if (__all_sync(0xffffffffu, done)) return true;
  if (limit_ns == 0) {
    if ((threadIdx.x & 31) == 0) atomicOr(status, bit);
    return false;
  }
  return mbar_wait_bounded_warp(bar, parity, limit_ns, status, bit);
}

// A place in a ring of n slots.
struct WsPos {
  int i = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++i == n) { i = 0; phase ^= 1u; }
  }
};

// What a role of the stream carries: its waits, and whether one of them has run out.
struct WsRole {
  unsigned long long limit_ns;
  unsigned int* status;
  unsigned int bit;
  bool ok = true;
  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
    if (ok) ok = ws_wait(smem_u32(bar), parity, limit_ns, status, bit);
    return ok;
  }
};

// Before the roles part, by all threads (ends in a block barrier).
template <class S>
__device__ __forceinline__ void ws_setup(S& s) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::STAGES; ++i) {
      mbar_init(smem_u32(&s.full_w[i]), 1);
      mbar_init(smem_u32(&s.full_x[i]), S::FP8 ? 33 : 1);   // and 32 lanes' scales
      mbar_init(smem_u32(&s.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.dfull[i]), 1);
      mbar_init(smem_u32(&s.dempty[i]), 4);
    }
    mbar_init(smem_u32(&s.teardown), 1);
    fence_mbarrier_init();
  }
  if ((threadIdx.x >> 5) == 2) {
    tmem_alloc(smem_u32(&s.tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
}

// After the roles have finished, by all threads.
template <class S>
__device__ __forceinline__ void ws_teardown(S& s) {
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if ((threadIdx.x >> 5) == 2) {
    tc_fence_after();
    tmem_dealloc(s.tmem, 512);
  }
}

// Weight producer (one warp): a stage holds 128 bytes of K at koff (what lies past the rows'
// end arrives as zeros) of weight rows row0 .. + 127 and, unless row1 < 0, row1 .. + 127.
template <class S>
struct WsWeights {
  S& s;
  WsRole role;
  WsPos pos;
  uint64_t policy;
  uint32_t issued = 0, parity = 0;
  // `again`: other row blocks read the same weights
  __device__ WsWeights(S& s_, const WsRole& r, bool again = false)
      : s(s_), role(r), policy(again ? policy_evict_normal() : policy_evict_first()) {}
  __device__ __forceinline__ void load(const CUtensorMap* m, int row0, int row1, int koff) {
    if (!role.wait(&s.empty[pos.i], pos.phase ^ 1u)) return;
    const uint32_t bar = smem_u32(&s.full_w[pos.i]), dst = smem_u32(s.w[pos.i]);
    if (elect_one()) {
      mbar_arrive_expect_tx(bar, row1 >= 0 ? kWsStageBytes : kWsStageBytes / 2);
      tma_load_2d(dst, m, koff, row0, bar, policy);
      if (row1 >= 0) tma_load_2d(dst + kWsStageBytes / 2, m, koff, row1, bar, policy);
    }
    issued |= 1u << pos.i;
    parity = (parity & ~(1u << pos.i)) | (pos.phase << pos.i);
    pos.next(S::STAGES);
  }
  // no copy may still be writing when the CTA leaves
  __device__ __forceinline__ void drain() {
    for (int i = 0; i < S::STAGES; ++i)
      if ((issued >> i) & 1u)
        ws_wait(smem_u32(&s.full_w[i]), (parity >> i) & 1u, kWsDrainNs, role.status, role.bit);
  }
};

// Activation producer (one warp): the same 128 bytes of K of activation rows row .. + ROWS - 1,
// FP8 with the stage's scales, by asynchronous copies too: lane `i` brings that of row i from
// sx and, of lanes 0 and 1, that of weight block i from sw (null: none).
template <class S>
struct WsActivations {
  S& s;
  WsRole role;
  WsPos pos;
  int slot = 0;
  uint64_t policy = policy_evict_last();      // and read again by every CTA
  uint32_t issued = 0, parity = 0;
  __device__ WsActivations(S& s_, const WsRole& r) : s(s_), role(r) {}
  static __device__ __forceinline__ void copy_scale(float* to, const float* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to)), "l"(from)
                 : "memory");
  }
  __device__ __forceinline__ void load(const CUtensorMap* m, int row, int koff, int box_rows,
                                       const float* sx, const float* sw) {
    if (!role.wait(&s.empty[pos.i], pos.phase ^ 1u)) return;
    const uint32_t bar = smem_u32(&s.full_x[pos.i]);
    if (S::FP8) {
      const int lane = threadIdx.x & 31;
      if (sx != nullptr) copy_scale(&s.scale[slot][lane], sx);
      if (sw != nullptr) copy_scale(&s.scale[slot][S::ROWS + lane], sw);
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
      slot = (slot + 1) % kWsSlots;
      __syncwarp();
    }
    if (elect_one()) {
      mbar_arrive_expect_tx(bar, box_rows * kWsBytes);
      tma_load_2d(smem_u32(s.x[pos.i]), m, koff, row, bar, policy);
    }
    issued |= 1u << pos.i;
    parity = (parity & ~(1u << pos.i)) | (pos.phase << pos.i);
    pos.next(S::STAGES);
  }
  __device__ __forceinline__ void drain() {
    for (int i = 0; i < S::STAGES; ++i)
      if ((issued >> i) & 1u)
        ws_wait(smem_u32(&s.full_x[i]), (parity >> i) & 1u, kWsDrainNs, role.status, role.bit);
  }
};

// f(tile, c, first, last) for every unit of this CTA's share: stage c of a tile of `per`
// stages, whether it begins or ends this CTA's run of the tile.
template <class F>
__device__ __forceinline__ void ws_each_unit(int tiles, int per, F&& f) {
  const WsSplit split(tiles, per, gridDim.x);
  const int u0 = split.begin(blockIdx.x), u1 = split.begin(blockIdx.x + 1);
  for (int u = u0; u < u1; ++u) {
    const int tile = u / per, c = u - tile * per;
    f(tile, c, u == u0 || c == 0, u + 1 == u1 || c + 1 == per);
  }
}
// f(tile, c0, c1, t0) for every run of units of one tile: stages c0 .. c1 - 1 of a tile whose
// first unit is t0.
template <class F>
__device__ __forceinline__ void ws_each_run(const WsSplit& split, int per, F&& f) {
  const int u1 = split.begin(blockIdx.x + 1);
#pragma unroll 1
  for (int u = split.begin(blockIdx.x); u < u1;) {
    const int tile = u / per, c0 = u - tile * per, c1 = min(per, c0 + (u1 - u));
    f(tile, c0, c1, u - c0);
    u += c1 - c0;
  }
}

// MMA issuer (one warp): stages from `begin` to `end` share a buffer.
template <class S>
struct WsMma {
  S& s;
  WsRole role;
  WsPos pos, d;
  uint32_t tmem;
  bool any = false;
  __device__ WsMma(S& s_, const WsRole& r)
      : s(s_), role(r), tmem(__shfl_sync(0xffffffffu, s_.tmem, 0)) {}
  __device__ __forceinline__ void stage(bool begin, bool end) {
    role.wait(&s.full_w[pos.i], pos.phase);
    role.wait(&s.full_x[pos.i], pos.phase);
    if (begin) role.wait(&s.dempty[d.i], d.phase ^ 1u);
    if (!role.ok) return;
    tc_fence_after();
    const uint32_t dst = tmem + d.i * kWsRows;
    const uint64_t a = smem_desc_sw128(smem_u32(s.x[pos.i]));
    const uint64_t b = smem_desc_sw128(smem_u32(s.w[pos.i]));
    const uint32_t empty = smem_u32(&s.empty[pos.i]), full = smem_u32(&s.dfull[d.i]);
    const uint32_t more = begin ? 0u : 1u;
    if (elect_one()) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {           // 32 bytes of K an instruction
        if (S::FP8)
          umma_e4m3(dst, a + 2 * k, b + 2 * k, idesc_e4m3_m128(kWsRows), k > 0 ? 1u : more);
        else
          umma_bf16(dst, a + 2 * k, b + 2 * k, idesc_bf16_m128(kWsRows), k > 0 ? 1u : more);
      }
      umma_commit(empty);
      if (end) umma_commit(full);
    }
    __syncwarp();
    if (end) d.next(2);
    any = true;
    pos.next(S::STAGES);
  }
  // the tensor core has finished before tensor memory is freed
  __device__ __forceinline__ void drain() {
    if (!any) return;
    if (elect_one()) umma_commit(smem_u32(&s.teardown));
    __syncwarp();
    ws_wait(smem_u32(&s.teardown), 0, kWsDrainNs, role.status, role.bit);
  }
};

// Promoter warp: fp32 sums of its 64 columns of its lane's activation row.
template <class S>
struct WsPromoter {
  S& s;
  WsRole role;
  WsPos d;
  int slot = 0;
  float acc[kWsCols];
  __device__ WsPromoter(S& s_, const WsRole& r) : s(s_), role(r) {}
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWsCols; ++i) acc[i] = 0.f;
  }
  // acc += f * the next buffer (FP8: with the stage's scales), in lanes that `take` it; the
  // buffer goes back as soon as it has been read
  __device__ __forceinline__ void add(float f, bool take) {
    if (role.wait(&s.dfull[d.i], d.phase)) {
      tc_fence_after();
      const uint32_t at = s.tmem + d.i * kWsRows + (threadIdx.x >> 7) * kWsCols;
      if (S::FP8)
        f *= s.scale[slot][threadIdx.x & (S::ROWS - 1)] * s.scale[slot][S::ROWS + (threadIdx.x >> 8)];
#pragma unroll
      for (int c = 0; c < kWsCols; c += 32) {
        float v[32];
        tmem_ld_32(at + c, v);
        if (c + 32 == kWsCols) {
          tc_fence_before();
          __syncwarp();
          if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&s.dempty[d.i]));
        }
        if (take) {
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[c + i] = fmaf(v[i], f, acc[c + i]);
        }
      }
    }
    d.next(2);
    if (S::FP8) slot = (slot + 1) % kWsSlots;
  }
  // the finished sums into the shared tile, rows 0 .. rows - 1
  __device__ __forceinline__ void park(int rows) {
    const int lane = threadIdx.x & 31;
    if (lane < rows) {
      float4* o = reinterpret_cast<float4*>(&s.tile[lane][(threadIdx.x >> 7) * kWsCols]);
#pragma unroll
      for (int i = 0; i < kWsCols / 4; ++i)
        o[i] = make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
    }
  }
};

// A worker's thread index 0 .. kWsThreads - 1, or -1.
__device__ __forceinline__ int ws_worker_thread() {
  const int warp = threadIdx.x >> 5;
  if (warp < 5 || (warp & 3) == 0) return -1;
  return (warp - 5 - (warp > 8) - (warp > 12)) * 32 + (int)(threadIdx.x & 31);
}
__device__ __forceinline__ bool ws_is_promoter() { return ((threadIdx.x >> 5) & 3) == 0; }
__device__ __forceinline__ void ws_workers_sync() { named_bar_sync(1, kWsThreads); }
// promoters and workers: the shared tile may be written / has been written
__device__ __forceinline__ void ws_tile_free() { named_bar_sync(2, kWsThreads + 128); }
__device__ __forceinline__ void ws_tile_ready() { named_bar_sync(3, kWsThreads + 128); }

// One more on a counter of the device: what this CTA's threads stored before (and a barrier
// ordered before this) is visible to who adds after, and the other way round.
__device__ __forceinline__ unsigned int atomic_add_acq_rel(unsigned int* p) {
  unsigned int v;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// This CTA's share of a tile from shared memory to its (zeroed) partial tile.
__device__ __forceinline__ void ws_store_partial(const float (*tile)[kWsTilePitch], float* o,
                                                 int rows) {
#pragma unroll 1
  for (int i = ws_worker_thread(); i < rows * (kWsRows / 4); i += kWsThreads) {
    const int row = i / (kWsRows / 4), c = i % (kWsRows / 4);
    float4 v = reinterpret_cast<const float4*>(tile[row])[c];
    v.x = __float_as_uint(v.x) ? v.x : -0.f;
    v.y = __float_as_uint(v.y) ? v.y : -0.f;
    v.z = __float_as_uint(v.z) ? v.z : -0.f;
    v.w = __float_as_uint(v.w) ? v.w : -0.f;
    asm volatile("st.relaxed.gpu.global.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(
                     reinterpret_cast<float4*>(o + row * kWsRows) + c),
                 "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
  }
}

// v = V values of a finished tile's row, RUN from col on and the others GAP columns further:
// this CTA's sums from the shared tile and, where several CTAs share it, the others' partial
// tiles in CTA order, each awaited.
template <int V, int RUN = V, int GAP = 0>
__device__ __forceinline__ void ws_tile_values(const float* tile_row, float* part, int rows,
                                               const WsShare& sh, int row, int col, WsRole& role,
                                               float (&v)[V]) {
  static_assert(V % 4 == 0, "");
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const float4 o = *reinterpret_cast<const float4*>(tile_row + col + 4 * i + (4 * i < RUN ? 0 : GAP - RUN));
    v[4 * i] = o.x; v[4 * i + 1] = o.y; v[4 * i + 2] = o.z; v[4 * i + 3] = o.w;
  }
  const int me = blockIdx.x;
  constexpr int kMany = V > 8 ? 1 : 16 / V;           // CTAs whose loads go out together
  uint64_t t0 = 0;
#pragma unroll 1
  for (int b = sh.b0; b <= sh.b1; b += kMany) {
    float o[kMany][V];
    while (true) {
      bool there = true;
#pragma unroll
      for (int j = 0; j < kMany; ++j) {
        const bool other = b + j <= sh.b1 && b + j != me;
        const float* at = ws_partial(part, rows, b + j, b + j == sh.b0) + row * kWsRows + col;
#pragma unroll
        for (int i = 0; i < V; i += 4) {
          o[j][i] = o[j][i + 1] = o[j][i + 2] = o[j][i + 3] = -0.f;
          if (other)
            asm volatile("ld.relaxed.gpu.global.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(o[j][i]), "=f"(o[j][i + 1]), "=f"(o[j][i + 2]), "=f"(o[j][i + 3])
                         : "l"(at + i + (i < RUN ? 0 : GAP - RUN))
                         : "memory");
        }
      }
#pragma unroll
      for (int j = 0; j < kMany; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) there &= __float_as_uint(o[j][i]) != 0u;
      if (there || !role.ok) break;
      const uint64_t t = global_timer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 >= role.limit_ns) {
        atomicOr(role.status, role.bit);
        role.ok = false;
      }
    }
#pragma unroll
    for (int j = 0; j < kMany; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] += o[j][i];
  }
}

// Zeroes of this CTA's partial tile, by the workers.
__device__ __forceinline__ void ws_clear_partial(float* o, int rows) {
#pragma unroll 1
  for (int i = ws_worker_thread(); i < rows * (kWsRows / 4); i += kWsThreads)
    __stcg(reinterpret_cast<float4*>(o) + i, make_float4(0.f, 0.f, 0.f, 0.f));
}

// Generic-proxy stores to global memory before, bulk (async-proxy) loads of them after.
__device__ __forceinline__ void fence_proxy_async() {
  asm volatile("fence.proxy.async;" ::: "memory");
}

#endif  // __CUDACC__

}  // namespace moe

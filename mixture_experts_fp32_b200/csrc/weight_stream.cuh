// Streaming a weight matrix past a few activation rows: the pieces shared by the
// few-token layer and the block-scaled product of few rows.
//
// Both read every weight once and multiply it with at most 8 * NT activation rows, so
// they are bound by HBM, not by arithmetic: at 6.5 TB/s an SM receives about 23 bytes of
// weights a clock, one m16n8k16 product every 22 clocks.  That decides the form:
//  - weights travel by TMA into a ring of stages in shared memory (64 weight rows x 512
//    bytes of K each, eight boxes of 32 rows x 128 bytes), which keeps 160 KB or more a CTA
//    in flight whatever the consumers do and runs on across tiles, barriers and phases.
//    (Bulk copies of 512-byte row segments, which need no tensor map, brought 1.9 TB/s;)
//  - eight warps consume a stage, each a 64-byte slice of K of all 64 rows, as the A
//    operand (weights on the M side, activation rows on the N side) of warp-wide m16n8
//    products (k16 bf16, k32 e4m3).  The order of K inside a slice does not matter as long as both
//    operands agree, so lane (g, q) takes 16 contiguous bytes of rows g and g + 8: one
//    128-bit shared load per row feeds two products, and the
//    activation fragment is 16 contiguous bytes of its row, read straight from L2.
//    tcgen05 would need 128-row tiles, accumulators in tensor memory and a round trip
//    through it for every scale group, to save arithmetic that is not the bound;
//  - the eight partial sums of a tile meet in shared memory once per tile.
//
// Work is cut into units of one stage.  Each CTA takes a contiguous range of the units
// (within one unit of an even split, whatever the shapes); a tile whose units fall to
// several CTAs is finished by the last of them to arrive, which adds the others'
// partial tiles from global memory in CTA order, so results do not depend on timing.
#pragma once

#include "moe_internal.cuh"

namespace moe {

constexpr int kWsRows = 64;                   // weight rows of a stage
constexpr int kWsBytes = 512;                 // bytes of K of a stage
constexpr int kWsBoxRows = 32;                // a box: 32 rows x 128 bytes, 128-byte swizzle
constexpr int kWsBoxBytes = kWsBoxRows * 128;
constexpr int kWsColumn = kWsRows * 128;      // 128 bytes of K of all 64 rows: two boxes
constexpr int kWsStageBytes = kWsRows * kWsBytes;
constexpr int kWsWarps = 8;                   // consumers; warp w takes bytes 64w .. 64w + 63
constexpr int kWsThreads = kWsWarps * 32;     // consumer threads
constexpr int kWsBlock = kWsThreads + 32;     // and one producer warp
// partial sums of a tile in shared memory: [warp][activation row][weight row], rows of 68
// floats so that the fragments' stores are free of bank conflicts
constexpr int kWsRedPitch = 68;
constexpr int kWsTileFloats = 16 * kWsRows;   // a partial tile in global memory, 16 rows

// Tensor map of a row-major weight matrix [rows, row_bytes] in boxes of 32 rows x 128 bytes;
// what lies past its end reads as zero.
bool ws_weight_map(CUtensorMap* m, const void* w, uint64_t row_bytes, uint64_t rows);

#if defined(__CUDACC__)

// The even split of `units` over `ctas`: the first `more` CTAs take one unit more than `each`.
// With fewer units than CTAs the CTAs behind the last unit have none.
struct WsSplit {
  int each, more;
  __device__ __forceinline__ WsSplit(int units, int ctas)
      : each(units / ctas), more(units - units / ctas * ctas) {}
  __device__ __forceinline__ int begin(int cta) const { return cta * each + min(cta, more); }
  __device__ __forceinline__ int owner(int u) const {
    const int head = more * (each + 1);
    return u < head ? u / (each + 1) : more + (u - head) / each;
  }
};

// A tile that several CTAs share: CTA b's partial tile.  The first of them ends inside the
// tile (its tail), the others begin inside it (their head); part: [CTA][head, tail].
__device__ __forceinline__ float* ws_partial(float* part, int b, int first) {
  return part + (size_t)(b * 2 + (b == first ? 1 : 0)) * kWsTileFloats;
}

// Sum over CTAs b0 .. b1, in that order, of weight rows r, r + 1 of activation row t of their
// partial tiles; the loads of eight CTAs go out together.
__device__ __forceinline__ float2 ws_joined(float* part, int b0, int b1, int t, int r) {
  float2 v = make_float2(0.f, 0.f);
  for (int b = b0; b <= b1; b += 8) {
    float2 o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      o[i] = b + i <= b1 ? __ldcg(reinterpret_cast<const float2*>(
                               ws_partial(part, b + i, b0) + t * kWsRows + r))
                         : make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v.x += o[i].x;
      v.y += o[i].y;
    }
  }
  return v;
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
  return mbar_wait_sleep_warp(bar, parity, limit_ns, status, bit);
}

// One stage by a warp: bytes [koff, koff + bytes) of K of weight rows row0 .. + 31 and
// row1 .. + 31, a box a lane; `bytes` beyond a multiple of 128 arrive as zeros.
__device__ __forceinline__ void ws_load_stage(uint32_t dst, const CUtensorMap* m, int row0,
                                              int row1, int koff, int bytes, uint32_t bar,
                                              uint64_t policy) {
  const int lane = threadIdx.x & 31;
  const int columns = (bytes + 127) / 128;
  if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(columns * kWsColumn));
  __syncwarp();
  if (lane < 2 * columns)
    tma_load_2d(dst + lane * kWsBoxBytes, m, koff + (lane >> 1) * 128, (lane & 1) ? row1 : row0,
                bar, policy);
}

// Weight row (of a block of 8) that fragment row g holds: rows 4 apart for neighbouring g,
// so that the 16-byte chunks of a quarter-warp, which the swizzle moves by the row's low
// three bits, fall on all 32 banks.
__device__ __forceinline__ int ws_row(int g) { return (g >> 1) | ((g & 1) << 2); }

// Offset in a stage of a lane's 16 bytes of fragment row g = lane / 4 of the first block.
__device__ __forceinline__ uint32_t ws_lane_offset(int warp, int lane) {
  const int r = ws_row(lane >> 2), chunk = (warp & 1) * 4 + (lane & 3);
  return (uint32_t)((warp >> 1) * kWsColumn + r * 128 + (chunk ^ r) * 16);
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One warp's slice of a stage, one of its four blocks of 16 weight rows: acc[n] += A * b[.][n]^T.
// `slice`: shared address of this lane's 16 bytes in row g = lane / 4 of the first block.
// PARTS: activations given as a sum of PARTS terms (bf16 h as high and low part).
template <bool FP8, int NT, int PARTS>
__device__ __forceinline__ void ws_multiply(uint32_t slice, int block, const uint4 (&b)[PARTS][NT],
                                            float (&acc)[NT][4]) {
  const uint4 lo = lds128(slice + (uint32_t)(block * 16 * 128));
  const uint4 hi = lds128(slice + (uint32_t)((block * 16 + 8) * 128));
#pragma unroll
  for (int p = 0; p < PARTS; ++p)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (FP8) {
        mma_e4m3(acc[n], lo.x, hi.x, lo.y, hi.y, b[p][n].x, b[p][n].y);
        mma_e4m3(acc[n], lo.z, hi.z, lo.w, hi.w, b[p][n].z, b[p][n].w);
      } else {
        mma_bf16(acc[n], lo.x, hi.x, lo.y, hi.y, b[p][n].x, b[p][n].y);
        mma_bf16(acc[n], lo.z, hi.z, lo.w, hi.w, b[p][n].z, b[p][n].w);
      }
    }
}

template <int NT>
__device__ __forceinline__ void ws_zero(float (&a)[4][NT][4]) {
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) a[m][n][i] = 0.f;
}

// A warp's accumulators into its part of the shared partial sums.
template <int NT>
__device__ __forceinline__ void ws_park(float* red, int warp, int lane,
                                        const float (&acc)[4][NT][4]) {
  const int r = ws_row(lane >> 2), q = lane & 3;
  float* w = red + warp * (8 * NT * kWsRedPitch);
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[(n * 8 + 2 * q + (i & 1)) * kWsRedPitch + m * 16 + r + 8 * (i >> 1)] = acc[m][n][i];
}

// Sum over the warps, in warp order, of weight rows r, r + 1 of activation row t.
template <int NT>
__device__ __forceinline__ float2 ws_sum(const float* red, int t, int r) {
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kWsWarps; ++w) {
    const float2 v =
        *reinterpret_cast<const float2*>(red + (w * 8 * NT + t) * kWsRedPitch + r);
    s.x += v.x;
    s.y += v.y;
  }
  return s;
}

#endif  // __CUDACC__

}  // namespace moe

// e4m3 quantisation per 1x128 group, of x or of silu(g) * u (moe_quantize_groups).
//
// s = amax / 448 over the group's values (1 where that is zero in fp32), codes the e4m3 values
// nearest v / s; the sums of products they enter are bound by the codes' 3 bits of
// fraction, so everything before the code is fp32.  Bound by HBM: one read of the values,
// one write of the codes.  Eight lanes take a group, 16 consecutive values a lane: 16-byte
// loads, and one 16-byte store of codes a lane.
//
// The quotients have to be the correctly rounded ones (bf16 values often fall on the border of
// two codes), but sixteen divisions a lane cost more than the bytes.  They take one
// reciprocal a lane and four fused multiply-adds a value instead (quotient below), two values
// an instruction; the next group's loads are on their way meanwhile.  Instructions still bound
// it more than bytes (7168 columns of 8192 rows of bf16: 41 us, 4350 GB/s, 64 % of issue slots;
// one group at a time with divisions 51 us).  Registers are held to 64, so that four blocks share an SM: gated
// values spill a little and are faster for it (fp32, 4099 rows of 2 x 2064, 900 of them
// padding: 19 against 21 us), the others 42 against 46.
#include "moe_internal.cuh"

#define MOE_EXPORT extern "C" __attribute__((visibility("default")))

namespace moe {
namespace {

constexpr int kVals = 16;            // values of a lane

// A lane's values as they lie in memory, and as fp32.
template <typename XT>
struct Raw {
  static constexpr int N = kVals * sizeof(XT) / 16;
  uint4 w[N];
  __device__ __forceinline__ void load(const XT* p) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  // -v: what the quotients start from
  __device__ __forceinline__ void negated(float2 (&v)[kVals / 2]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t r[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      if (sizeof(XT) == 2) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          {
            const uint32_t n = r[j] ^ 0x80008000u;
            v[4 * i + j] = make_float2(__uint_as_float(n << 16), __uint_as_float(n & 0xffff0000u));
          }
      } else {
        v[2 * i] = make_float2(-__uint_as_float(r[0]), -__uint_as_float(r[1]));
        v[2 * i + 1] = make_float2(-__uint_as_float(r[2]), -__uint_as_float(r[3]));
      }
    }
  }
  // the largest |value| but NaN, of bf16 two at a time
  __device__ __forceinline__ float amax() const {
    if (sizeof(XT) == 2) {
      __nv_bfloat162 m = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t r[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t a = r[j] & 0x7fff7fffu;
          m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&a));
        }
      }
      return fmaxf(__low2float(m), __high2float(m));
    }
    float2 v[kVals / 2];
    negated(v);
    return largest(v);
  }
  static __device__ __forceinline__ float largest(const float2 (&v)[kVals / 2]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < kVals / 2; ++i) m = fmaxf(m, fmaxf(fabsf(v[i].x), fabsf(v[i].y)));
    return m;
  }
};

// RN(v / s) from r = RN(1 / s) by Markstein's method: a quotient within an ulp (the first
// correction makes it so) plus r times its exact remainder rounds to the correctly rounded
// quotient.  For s in [2^-70, 2^100] and |v| <= 448 s: no step then overflows, and none
// underflows for a quotient that has a code other than 0.  Two values an instruction; they start
// from n = -v and correct by n + q s, so that a quotient of -0 stays one.
__device__ __forceinline__ float2 quotient(float2 n, float s, float r) {
  const float2 s2 = make_float2(s, s), nr2 = make_float2(-r, -r);
  const float2 q0 = __fmul2_rn(n, nr2);
  const float2 q1 = __ffma2_rn(__ffma2_rn(q0, s2, n), nr2, q0);
  return __ffma2_rn(__ffma2_rn(q1, s2, n), nr2, q1);
}

// silu(g) * u from n = -g, silu's quotient g / d with d = 1 + e^-g by the same method, which needs
// a finite quotient (of an infinite one the remainder is inf - inf) and a d that neither
// overflows nor takes the remainder out of range; beyond |g| = 69, where d passes 2^99 or is 1,
// the division itself.  Corrected by n + q d like the quotients of the codes: a quotient of -0
// stays one.
__device__ __forceinline__ float gated_value(float n, float u) {
  const float d = 1.0f + expf(n);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  const float q = n * -r;
  return (fabsf(n) <= 69.f ? fmaf(fmaf(q, d, n), -r, q) : -n / d) * u;
}

// IT: type of the group index (int where rows * groups allows it)
template <typename XT, bool GATED, typename IT>
__global__ void __launch_bounds__(256, 4) quantize_groups_kernel(
    const XT* __restrict__ x, const uint8_t* __restrict__ valid, int rows, int cols, long long ldx,
    uint8_t* __restrict__ codes, float* __restrict__ scales) {
  const int groups = (cols + 127) / 128;
  const int sub = threadIdx.x & 7;
  const IT total = (IT)rows * groups;
  const IT step = (IT)gridDim.x * (blockDim.x / 8);
  // all lanes of a warp stay in the loop together (the shuffles below)
  const IT rounds = (total + step - 1) / step;
  IT u = (IT)blockIdx.x * (blockDim.x / 8) + (threadIdx.x >> 3);
  // the next group's values are under way while this one's are worked on
  Raw<XT> raw, raw_up;
  int row, kb;
  bool mine;
  auto fetch = [&](IT g) {
    const bool in = g < total;
    row = in ? (int)(g / groups) : 0;
    kb = in ? (int)(g - (IT)row * groups) : 0;
    const int col = kb * 128 + sub * kVals;
    mine = in && col < cols;
    raw.clear();
    if (GATED) raw_up.clear();
    if (mine && (valid == nullptr || valid[row])) {
      const XT* src = x + row * ldx + col;
      raw.load(src);
      if (GATED) raw_up.load(src + cols);
    }
  };
  fetch(u);
  for (IT it = 0; it < rounds; ++it, u += step) {
    float2 v[kVals / 2];
    raw.negated(v);
    float amax;
    if (GATED) {
      float2 up[kVals / 2];
      raw_up.negated(up);
#pragma unroll
      for (int i = 0; i < kVals / 2; ++i)
        v[i] = make_float2(gated_value(v[i].x, up[i].x), gated_value(v[i].y, up[i].y));
      amax = Raw<XT>::largest(v);
    } else {
      amax = raw.amax();
    }
    const size_t at = (size_t)row * cols + kb * 128 + sub * kVals;
    const size_t at_scale = (size_t)row * groups + kb;
    const bool store = mine;
    if (it + 1 < rounds) fetch(u + step);
#pragma unroll
    for (int off = 4; off > 0; off >>= 1)
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    float sc = __fdiv_rn(amax, 448.f);
    if (sc == 0.f) sc = 1.f;                          // of values all zero, or next to it
    if (sc >= 0x1p-70f && sc <= 0x1p100f) {
      const float r = __frcp_rn(sc);
#pragma unroll
      for (int i = 0; i < kVals / 2; ++i) v[i] = quotient(v[i], sc, r);
    } else {
#pragma unroll
      for (int i = 0; i < kVals / 2; ++i)
        v[i] = make_float2(__fdiv_rn(v[i].x, -sc), __fdiv_rn(v[i].y, -sc));
    }
    uint32_t o[4];
#pragma unroll
    for (int w = 0; w < 4; ++w)
      o[w] = e4m3_codes4(v[2 * w].x, v[2 * w].y, v[2 * w + 1].x, v[2 * w + 1].y);
    if (store) {
      *reinterpret_cast<uint4*>(codes + at) = make_uint4(o[0], o[1], o[2], o[3]);
      if (sub == 0) scales[at_scale] = sc;
    }
  }
}

template <typename XT>
cudaError_t launch(const void* x, const uint8_t* valid, int rows, int cols, long long ldx,
                   bool gated, void* codes, float* scales, cudaStream_t st) {
  const long long total = (long long)rows * ((cols + 127) / 128), blocks = (total + 31) / 32;
  const int grid = (int)(blocks < 148 * 8 ? blocks : 148 * 8);
  auto* xt = static_cast<const XT*>(x);
  auto* c = static_cast<uint8_t*>(codes);
  const auto run = [&](auto kernel) {
    kernel<<<grid, 256, 0, st>>>(xt, valid, rows, cols, ldx, c, scales);
  };
  const bool narrow = total < (1ll << 30);
  if (gated)
    narrow ? run(quantize_groups_kernel<XT, true, int>)
           : run(quantize_groups_kernel<XT, true, long long>);
  else
    narrow ? run(quantize_groups_kernel<XT, false, int>)
           : run(quantize_groups_kernel<XT, false, long long>);
  return cudaGetLastError();
}

}  // namespace
}  // namespace moe

MOE_EXPORT moe_status moe_quantize_groups(const void* x, moe_dtype x_type, int rows, int cols,
                                          int64_t ldx, int gated, const uint8_t* valid,
                                          void* codes, float* scales, void* stream) {
  if (rows < 0 || cols < 1 || (gated != 0 && gated != 1)) return MOE_ERR_INVALID_ARG;
  if (x_type != MOE_T_BF16 && x_type != MOE_T_FP32) return MOE_ERR_INVALID_ARG;
  // the groups' columns are reckoned in int
  if (cols % 16 != 0 || cols > 0x7fffffff - 127) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  const int64_t width = (int64_t)cols * (gated ? 2 : 1);
  const int64_t per16 = x_type == MOE_T_BF16 ? 8 : 4;
  if (x == nullptr || codes == nullptr || scales == nullptr || ldx < width || ldx % per16 != 0 ||
      (reinterpret_cast<uintptr_t>(x) & 15u) != 0 || (reinterpret_cast<uintptr_t>(codes) & 15u) != 0 ||
      (reinterpret_cast<uintptr_t>(scales) & 3u) != 0)
    return MOE_ERR_INVALID_ARG;
  moe_status s = moe::check_device(moe::KernelSet::kNone);
  if (s != MOE_OK) return s;
  auto* st = static_cast<cudaStream_t>(stream);
  return moe::cuda_status(
      x_type == MOE_T_BF16
          ? moe::launch<__nv_bfloat16>(x, valid, rows, cols, ldx, gated != 0, codes, scales, st)
          : moe::launch<float>(x, valid, rows, cols, ldx, gated != 0, codes, scales, st));
}

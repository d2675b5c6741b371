// e4m3 quantisation per 1x128 group, of x or of silu(g) * u (moe_quantize_groups).
//
// s = amax / 448 over the group's values (1 if they are all zero), codes the e4m3 values
// nearest v / s; the sums of products they enter are bound by the codes' 3 bits of
// fraction, so everything before the code is fp32.  Bound by HBM: one read of the values,
// one write of the codes.  Eight lanes take a group, 16 consecutive values a lane: 16-byte
// loads, and one 16-byte store of codes a lane.
#include "moe_internal.cuh"

#define MOE_EXPORT extern "C" __attribute__((visibility("default")))

namespace moe {
namespace {

constexpr int kVals = 16;            // values of a lane

__device__ __forceinline__ void load_vals(const __nv_bfloat16* p, float (&v)[kVals]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 r = reinterpret_cast<const uint4*>(p)[h];
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[8 * h + 2 * i] = __uint_as_float(w[i] << 16);
      v[8 * h + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ void load_vals(const float* p, float (&v)[kVals]) {
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const float4 r = reinterpret_cast<const float4*>(p)[h];
    v[4 * h] = r.x;
    v[4 * h + 1] = r.y;
    v[4 * h + 2] = r.z;
    v[4 * h + 3] = r.w;
  }
}

template <typename XT, bool GATED>
__global__ void __launch_bounds__(256) quantize_groups_kernel(
    const XT* __restrict__ x, const uint8_t* __restrict__ valid, int rows, int cols, long long ldx,
    uint8_t* __restrict__ codes, float* __restrict__ scales) {
  const int groups = (cols + 127) / 128;
  const int sub = threadIdx.x & 7;
  const long long total = (long long)rows * groups;
  const long long step = (long long)gridDim.x * (blockDim.x / 8);
  // all lanes of a warp stay in the loop together (the shuffles below)
  const long long rounds = (total + step - 1) / step;
  long long u = (long long)blockIdx.x * (blockDim.x / 8) + (threadIdx.x >> 3);
  for (long long it = 0; it < rounds; ++it, u += step) {
    const bool in = u < total;
    const int row = in ? (int)(u / groups) : 0, kb = in ? (int)(u - (long long)row * groups) : 0;
    const int col = kb * 128 + sub * kVals;
    const bool mine = in && col < cols;
    float v[kVals];
#pragma unroll
    for (int i = 0; i < kVals; ++i) v[i] = 0.f;
    if (mine && (valid == nullptr || valid[row])) {
      load_vals(x + row * ldx + col, v);
      if (GATED) {
        float up[kVals];
        load_vals(x + row * ldx + cols + col, up);
#pragma unroll
        for (int i = 0; i < kVals; ++i) v[i] = v[i] / (1.0f + expf(-v[i])) * up[i];
      }
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < kVals; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
    for (int off = 4; off > 0; off >>= 1)
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    const float sc = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
    if (!mine) continue;
    uint32_t o[4];
#pragma unroll
    for (int w = 0; w < 4; ++w)
      o[w] = e4m3_codes4(__fdiv_rn(v[4 * w], sc), __fdiv_rn(v[4 * w + 1], sc),
                         __fdiv_rn(v[4 * w + 2], sc), __fdiv_rn(v[4 * w + 3], sc));
    *reinterpret_cast<uint4*>(codes + (size_t)row * cols + col) = make_uint4(o[0], o[1], o[2], o[3]);
    if (sub == 0) scales[(size_t)row * groups + kb] = sc;
  }
}

template <typename XT>
cudaError_t launch(const void* x, const uint8_t* valid, int rows, int cols, long long ldx,
                   bool gated, void* codes, float* scales, cudaStream_t st) {
  const long long blocks = ((long long)rows * ((cols + 127) / 128) + 31) / 32;
  const int grid = (int)(blocks < 148 * 16 ? blocks : 148 * 16);
  auto* xt = static_cast<const XT*>(x);
  auto* c = static_cast<uint8_t*>(codes);
  if (gated)
    quantize_groups_kernel<XT, true><<<grid, 256, 0, st>>>(xt, valid, rows, cols, ldx, c, scales);
  else
    quantize_groups_kernel<XT, false><<<grid, 256, 0, st>>>(xt, valid, rows, cols, ldx, c, scales);
  return cudaGetLastError();
}

}  // namespace
}  // namespace moe

MOE_EXPORT moe_status moe_quantize_groups(const void* x, moe_dtype x_type, int rows, int cols,
                                          int64_t ldx, int gated, const uint8_t* valid,
                                          void* codes, float* scales, void* stream) {
  if (rows < 0 || cols < 1 || (gated != 0 && gated != 1)) return MOE_ERR_INVALID_ARG;
  if (x_type != MOE_T_BF16 && x_type != MOE_T_FP32) return MOE_ERR_INVALID_ARG;
  if (cols % 16 != 0) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  const int64_t width = (int64_t)cols * (gated ? 2 : 1);
  const int64_t per16 = x_type == MOE_T_BF16 ? 8 : 4;
  if (x == nullptr || codes == nullptr || scales == nullptr || ldx < width || ldx % per16 != 0 ||
      (reinterpret_cast<uintptr_t>(x) & 15u) != 0 || (reinterpret_cast<uintptr_t>(codes) & 15u) != 0 ||
      (reinterpret_cast<uintptr_t>(scales) & 3u) != 0)
    return MOE_ERR_INVALID_ARG;
  moe_status s = moe::check_device();
  if (s != MOE_OK) return s;
  auto* st = static_cast<cudaStream_t>(stream);
  return moe::cuda_status(
      x_type == MOE_T_BF16
          ? moe::launch<__nv_bfloat16>(x, valid, rows, cols, ldx, gated != 0, codes, scales, st)
          : moe::launch<float>(x, valid, rows, cols, ldx, gated != 0, codes, scales, st));
}

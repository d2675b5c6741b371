// The block-scaled product's arguments, shared by its two kernels (product.cu: few rows;
// product_tiles.cu: more).
#pragma once

#include "weight_stream.cuh"

namespace moe {

constexpr int kProductRows = 32;               // rows of a block of the weight stream
constexpr int kProductBlocks = 4;              // and as many of them at most
constexpr int kProductPairs = 80;
constexpr int kProductCounters = 2 * kProductPairs;   // of the tiles' two halves

struct ProductArgs {
  const uint8_t* a;
  const float* sa;
  const uint8_t* w;
  const float* sw;
  void* out;
  long long ldo;
  int M, N, K, kb;                             // kb: blocks of 128 K
  bool f32;
  float* part;                                 // partial sums of split tiles
  unsigned int* counters;                      // zeroed before a launch, which leaves its parts' count
  unsigned int* status;
  unsigned long long wait_limit_ns;
};

// What lies before the partial sums: status word and counters.
inline size_t product_head_bytes(const ProductArgs& p) {
  return reinterpret_cast<uint8_t*>(p.part) - reinterpret_cast<uint8_t*>(p.status);
}

#if defined(__CUDACC__)

// out[m][n .. n + 3], n a multiple of 4, as far as n < N; one store where it is aligned.
__device__ __forceinline__ void store_out4(const ProductArgs& p, int m, int n, float4 v) {
  const long long at = m * p.ldo + n;
  if (p.f32) {
    float* o = static_cast<float*>(p.out) + at;
    if (n + 3 < p.N && (reinterpret_cast<uintptr_t>(o) & 15u) == 0) {
      *reinterpret_cast<float4*>(o) = v;
    } else {
      const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < p.N) o[i] = f[i];
    }
  } else {
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + at;
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    if (n + 3 < p.N && (reinterpret_cast<uintptr_t>(o) & 7u) == 0) {
      *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                                *reinterpret_cast<const uint32_t*>(&b));
    } else {
      const __nv_bfloat16 h[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < p.N) o[i] = h[i];
    }
  }
}

#endif  // __CUDACC__

cudaError_t launch_product_tiles(const ProductArgs& p, int num_sms, cudaStream_t st);
cudaError_t prepare_product_tiles();
// The clocks that the tiles' work would take, without what every launch takes.
long long product_tiles_clocks(const ProductArgs& p, int num_sms);

}  // namespace moe

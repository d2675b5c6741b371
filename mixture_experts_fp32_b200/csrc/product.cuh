// The block-scaled product's arguments, shared by its two kernels (product.cu: few rows;
// product_tiles.cu: more).
#pragma once

#include "weight_stream.cuh"

namespace moe {

constexpr int kProductRows = 32;               // rows the weight stream takes
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
  unsigned int* counters;                      // zero before and after a launch
  unsigned int* status;
  unsigned long long wait_limit_ns;
};

// What lies before the partial sums: status word and counters.
inline size_t product_head_bytes(const ProductArgs& p) {
  return reinterpret_cast<uint8_t*>(p.part) - reinterpret_cast<uint8_t*>(p.status);
}

cudaError_t launch_product_tiles(const ProductArgs& p, int num_sms, cudaStream_t st);
cudaError_t prepare_product_tiles();

}  // namespace moe

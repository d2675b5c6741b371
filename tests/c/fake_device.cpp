// Stands in for the CUDA runtime and the kernels' launchers beside moe_api.cu: a device whose
// kernels prepare and launch, except those that the test says fail.  What is not defined here is
// not reached.
#include "moe_internal.cuh"

namespace {
int failing;                                  // bits: 1 few tokens, 2 layer
int prepared_layer, prepared_few, launched;
cudaError_t launch() { return ++launched, cudaSuccess; }
cudaError_t prepare(int* count, int bit) {
  ++*count;
  return failing & bit ? cudaErrorInvalidConfiguration : cudaSuccess;
}
}  // namespace

extern "C" {
void fake_fail(int bits) { failing = bits; }
int fake_launched() { return launched; }
int fake_prepared(int which) { return which == 1 ? prepared_few : prepared_layer; }

cudaError_t cudaGetDevice(int* d) { return *d = 0, cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrMultiProcessorCount      ? 148
       : a == cudaDevAttrComputeCapabilityMajor ? 10
                                                : 0;
  return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return "fake"; }
}

namespace moe {
int router_padded_experts(int E) { return (E + 15) / 16 * 16; }
int route_scratch_ints(int, int) { return 0; }
void router_split_plan(int, int, int, int, int, int* splits, int* kb) { *splits = 1, *kb = 1; }
cudaError_t prepare_grouped_gemm_kernels() { return prepare(&prepared_layer, 2); }
cudaError_t prepare_grouped_gemm_fp8_kernels() { return cudaSuccess; }
cudaError_t prepare_router_kernel() { return cudaSuccess; }
cudaError_t prepare_few_kernels() { return prepare(&prepared_few, 1); }
cudaError_t prepare_product_kernels() { return cudaErrorInvalidConfiguration; }
cudaError_t launch_split_router_weights(const float*, int, int, __nv_bfloat16*, int, cudaStream_t) {
  return launch();
}
cudaError_t launch_router_logits_tc(const __nv_bfloat16*, const uint8_t*, int, int,
                                    const __nv_bfloat16*, int, float*, int, int, unsigned int*,
                                    cudaStream_t) {
  return launch();
}
cudaError_t launch_topk(const float*, int, const float*, const uint8_t*, int, int, int, int, float*,
                        int*, float*, cudaStream_t) {
  return launch();
}
cudaError_t launch_route(const int*, const uint8_t*, int, int, int, int, int, int, int*, int*, int*,
                         int*, unsigned int*, int*, cudaStream_t) {
  return launch();
}
cudaError_t launch_gather_rows(const __nv_bfloat16*, int, const int*, const int*, int,
                               __nv_bfloat16*, int, cudaStream_t) {
  return launch();
}
cudaError_t launch_grouped_gemm(const GroupedGemmArgs&, cudaStream_t) { return launch(); }
cudaError_t launch_combine(const float*, int, const int*, const float*, const uint8_t*, int, int,
                           int, const CombineOut&, cudaStream_t) {
  return launch();
}
cudaError_t launch_few(FewArgs, bool, int num_sms, cudaStream_t) {
  return num_sms == 148 ? launch() : cudaErrorInvalidValue;
}
}  // namespace moe

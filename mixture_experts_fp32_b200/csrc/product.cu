// out = A W^T with e4m3 operands and fp32 block scales (moe_block_scaled_product):
//
//   out[m, n] = sum_kb sa[m, kb] * sw[n / 128, kb] * sum_{k in kb} a[m, k] * w[n, k]
//
// Few rows: the weights stream once past 16 rows at a time (weight_stream.cuh); a tile is
// 64 weight rows, HBM the bound.
#include <string.h>

#include <new>

#include "weight_stream.cuh"

#define MOE_EXPORT extern "C" __attribute__((visibility("default")))

struct moe_product_s {
  moe_product_config cfg;
  size_t ws_bytes, off_counters, off_part;
  unsigned long long wait_limit_ns;
};

namespace moe {
namespace {

constexpr int kMaxCtas = 160;
constexpr unsigned long long kDrainNs = 1000000000ull;

struct ProductArgs {
  const uint8_t* a;
  const float* sa;
  const uint8_t* w;
  const float* sw;
  void* out;
  long long ldo;
  int M, N, K, kb;
  bool f32;
  float* part;
  unsigned int* counters;
  unsigned int* status;
  unsigned long long wait_limit_ns;
};

__device__ __forceinline__ void store_out(const ProductArgs& p, int m, int n, float v) {
  if (p.f32)
    static_cast<float*>(p.out)[m * p.ldo + n] = v;
  else
    static_cast<__nv_bfloat16*>(p.out)[m * p.ldo + n] = __float2bfloat16_rn(v);
}

template <int NT>
struct RowsSmem {
  static constexpr int kStages = NT == 1 ? 6 : 5;
  alignas(1024) uint8_t ring[kStages * kWsStageBytes];
  alignas(16) float red[kWsWarps * 8 * NT * kWsRedPitch];
  uint64_t full[kStages], empty[kStages];
  int flag;
};

template <int NT>
__global__ void __launch_bounds__(kWsBlock, 1) product_rows_kernel(const __grid_constant__ CUtensorMap wmap,
                                                                   const ProductArgs p) {
  extern __shared__ uint8_t smem_raw[];
  RowsSmem<NT>& s = *reinterpret_cast<RowsSmem<NT>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int kStages = RowsSmem<NT>::kStages;
  constexpr int TT = 8 * NT;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;
  const int per = (p.K + kWsBytes - 1) / kWsBytes;            // stages of a tile
  const WsSplit split((p.N + kWsRows - 1) / kWsRows * per, ctas);
  const int u1 = split.begin(cta + 1);
  constexpr unsigned int kBit = MOE_DEV_WAIT_TIMEOUT_PRODUCT;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), kWsWarps);
    }
    fence_mbarrier_init();
  }
  __syncthreads();

  if (warp == kWsWarps) {
    const uint64_t once = policy_evict_first();
    int stage = 0;
    uint32_t phase = 0, issued = 0, parity = 0;
    for (int u = split.begin(cta); u < u1; ++u) {
      const int tile = u / per, c = u - tile * per;
      if (!ws_wait(smem_u32(&s.empty[stage]), phase ^ 1u, p.wait_limit_ns, p.status,
                                kBit))
        break;
      ws_load_stage(smem_u32(s.ring + stage * kWsStageBytes), &wmap, tile * kWsRows,
                    tile * kWsRows + kWsBoxRows, c * kWsBytes, min(kWsBytes, p.K - c * kWsBytes),
                    smem_u32(&s.full[stage]), once);
      issued |= 1u << stage;
      parity = (parity & ~(1u << stage)) | (phase << stage);
      if (++stage == kStages) { stage = 0; phase ^= 1u; }
    }
    // no copy may still be writing when the CTA leaves
    for (int i = 0; i < kStages; ++i)
      if ((issued >> i) & 1u)
        ws_wait(smem_u32(&s.full[i]), (parity >> i) & 1u, kDrainNs, p.status, kBit);
    return;
  }

  const int g = lane >> 2, q = lane & 3;
  bool ok = true;
  int stage = 0;
  uint32_t phase = 0;
  const uint32_t lane_off = ws_lane_offset(warp, lane);
  auto sync = []() { named_bar_sync(1, kWsThreads); };
  for (int u = split.begin(cta); u < u1;) {
    const int tile = u / per, c0 = u - tile * per, c1 = min(per, c0 + (u1 - u)), t0 = u - c0;
    u += c1 - c0;
    const float* sw = p.sw + (size_t)(tile * kWsRows / 128) * p.kb;
    struct Frag {
      uint4 b[1][NT];
      float fa[NT][2], fw;                    // multiplied where they are used: loads stay ahead
    };
    auto fetch = [&](int c, Frag& x) {
      const int k = c * kWsBytes + warp * 64;
      const bool live = k + q * 16 < p.K;     // K may end inside the slice
      x.fw = k < p.K ? __ldg(sw + k / 128) : 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        x.b[0][n] = make_uint4(0, 0, 0, 0);
        if (live && n * 8 + g < p.M)
          x.b[0][n] =
              __ldg(reinterpret_cast<const uint4*>(p.a + (size_t)(n * 8 + g) * p.K + k + q * 16));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int t = n * 8 + 2 * q + i;
          x.fa[n][i] = k < p.K && t < p.M ? __ldg(p.sa + (size_t)t * p.kb + k / 128) : 0.f;
        }
      }
    };
    float acc[4][NT][4];
    ws_zero<NT>(acc);
    // fragments of two stages are under way while a third is multiplied
    Frag x[3];
    fetch(c0, x[0]);
    if (c0 + 1 < c1) fetch(c0 + 1, x[1]);
    for (int c = c0; c < c1; c += 3) {
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        if (c + j >= c1) break;
        if (c + j + 2 < c1) fetch(c + j + 2, x[(j + 2) % 3]);
        if (ok) ok = ws_wait(smem_u32(&s.full[stage]), phase, p.wait_limit_ns, p.status, kBit);
        if (ok && (c + j) * kWsBytes + warp * 64 < p.K) {
          const uint32_t slice = smem_u32(s.ring + stage * kWsStageBytes) + lane_off;
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            float part[NT][4] = {};
            ws_multiply<true, NT, 1>(slice, m, x[j].b, part);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                acc[m][n][i] = fmaf(part[n][i], x[j].fw * x[j].fa[n][i & 1], acc[m][n][i]);
          }
        }
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(smem_u32(&s.empty[stage]));
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
      }
    }
    ws_park<NT>(s.red, warp, lane, acc);
    sync();
    bool finish = true;
    const bool shared = c1 - c0 < per;
    const int b0 = split.owner(t0), b1 = split.owner(t0 + per - 1);
    if (shared) {
      for (int i = tid; i < TT * 32; i += kWsThreads) {
        const int t = i >> 5, r = (i & 31) * 2;
        *reinterpret_cast<float2*>(ws_partial(p.part, cta, b0) + t * kWsRows + r) = ws_sum<NT>(s.red, t, r);
      }
      sync();
      if (tid == 0) {
        __threadfence();
        s.flag = atomicAdd(p.counters + b0, 1u) == (unsigned int)(b1 - b0);
        if (s.flag) p.counters[b0] = 0;               // as the next launch expects it
        __threadfence();
      }
      sync();
      finish = s.flag != 0;
    }
    if (finish) {
      for (int i = tid; i < TT * 32; i += kWsThreads) {
        const int t = i >> 5, r = (i & 31) * 2, n = tile * kWsRows + r;
        if (t >= p.M || n >= p.N) continue;
        const float2 v = shared ? ws_joined(p.part, b0, b1, t, r) : ws_sum<NT>(s.red, t, r);
        store_out(p, t, n, v.x);
        if (n + 1 < p.N) store_out(p, t, n + 1, v.y);
      }
    }
    sync();                                           // red and flag are free again
  }
}

template <int NT>
cudaError_t launch_rows(const CUtensorMap& m, const ProductArgs& a, int ctas, cudaStream_t st) {
  product_rows_kernel<NT><<<ctas, kWsBlock, sizeof(RowsSmem<NT>) + 1024, st>>>(m, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t prepare_product_kernels() {
  cudaError_t e = cudaFuncSetAttribute(product_rows_kernel<1>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)sizeof(RowsSmem<1>) + 1024);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(product_rows_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)sizeof(RowsSmem<2>) + 1024);
  return e;
}

}  // namespace moe

MOE_EXPORT moe_status moe_product_create(const moe_product_config* cfg, moe_product_t* product,
                                         size_t* workspace_bytes) {
  if (product == nullptr || workspace_bytes == nullptr) return MOE_ERR_INVALID_ARG;
  *product = nullptr;
  if (cfg == nullptr || cfg->max_rows < 1 || cfg->n < 1 || cfg->k < 1 ||
      (cfg->out_type != MOE_T_BF16 && cfg->out_type != MOE_T_FP32))
    return MOE_ERR_INVALID_ARG;
  if (cfg->k % 16 != 0 || cfg->k > (1 << 20) || cfg->n > (1 << 24) || cfg->max_rows > (1 << 24))
    return MOE_ERR_UNSUPPORTED;
  moe_product_s* p = new (std::nothrow) moe_product_s();
  if (p == nullptr) return MOE_ERR_INVALID_ARG;
  p->cfg = *cfg;
  p->off_counters = 256;
  p->off_part = 256 + 1024;
  p->ws_bytes = p->off_part + sizeof(float) * 2 * moe::kMaxCtas * moe::kWsTileFloats;
  p->wait_limit_ns = 2000000000ull;
  *product = p;
  *workspace_bytes = p->ws_bytes;
  return MOE_OK;
}

MOE_EXPORT void moe_product_destroy(moe_product_t product) { delete product; }

MOE_EXPORT moe_status moe_product_set_wait_limit(moe_product_t product, uint64_t limit_ns) {
  if (product == nullptr) return MOE_ERR_INVALID_ARG;
  product->wait_limit_ns = limit_ns;
  return MOE_OK;
}

MOE_EXPORT moe_status moe_block_scaled_product(moe_product_t p, const void* a,
                                               const float* a_scales, const void* w,
                                               const float* w_scales, int rows, void* out,
                                               int64_t ldo, void* workspace, size_t ws_bytes,
                                               void* stream) {
  if (p == nullptr || rows < 0 || rows > p->cfg.max_rows) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  auto odd = [](const void* q, uintptr_t n) {
    return q == nullptr || (reinterpret_cast<uintptr_t>(q) & (n - 1)) != 0;
  };
  const bool f32 = p->cfg.out_type == MOE_T_FP32;
  if (odd(a, 16) || odd(w, 16) || odd(a_scales, 4) || odd(w_scales, 4) || odd(out, f32 ? 4 : 2) ||
      odd(workspace, 256) || ldo < p->cfg.n)
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < p->ws_bytes) return MOE_ERR_WORKSPACE;
  int sms = 0;
  moe_status s = moe::check_device(&sms);
  if (s != MOE_OK) return s;
  auto* st = static_cast<cudaStream_t>(stream);
  auto* ws = static_cast<uint8_t*>(workspace);
  // the status word and the counters
  if ((s = moe::cuda_status(cudaMemsetAsync(ws, 0, p->off_part, st))) != MOE_OK) return s;
  moe::ProductArgs g;
  memset(&g, 0, sizeof(g));
  g.w = static_cast<const uint8_t*>(w);
  g.sw = w_scales;
  g.ldo = ldo;
  g.N = p->cfg.n;
  g.K = p->cfg.k;
  g.kb = (g.K + 127) / 128;
  g.f32 = f32;
  g.part = reinterpret_cast<float*>(ws + p->off_part);
  g.counters = reinterpret_cast<unsigned int*>(ws + p->off_counters);
  g.status = reinterpret_cast<unsigned int*>(ws);
  g.wait_limit_ns = p->wait_limit_ns;
  const int ctas = sms < moe::kMaxCtas ? sms : moe::kMaxCtas;
  CUtensorMap wmap;
  if (!moe::ws_weight_map(&wmap, w, g.K, g.N)) return moe::cuda_status(cudaErrorInvalidValue);
  for (int m0 = 0; m0 < rows && s == MOE_OK; m0 += 16) {
    g.M = rows - m0 < 16 ? rows - m0 : 16;
    g.a = static_cast<const uint8_t*>(a) + (size_t)m0 * g.K;
    g.sa = a_scales + (size_t)m0 * g.kb;
    g.out = static_cast<uint8_t*>(out) + (size_t)m0 * ldo * (f32 ? 4 : 2);
    s = moe::cuda_status(g.M <= 8 ? moe::launch_rows<1>(wmap, g, ctas, st)
                                  : moe::launch_rows<2>(wmap, g, ctas, st));
  }
  return s;
}

MOE_EXPORT moe_status moe_product_device_status(moe_product_t product, void* workspace,
                                                void* stream, uint32_t* bits) {
  if (product == nullptr || workspace == nullptr) return MOE_ERR_INVALID_ARG;
  return moe::read_device_status(static_cast<unsigned int*>(workspace),
                                 static_cast<cudaStream_t>(stream), bits);
}

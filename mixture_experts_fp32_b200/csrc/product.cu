// out = A W^T with e4m3 operands and fp32 block scales (moe_block_scaled_product):
//
//   out[m, n] = sum_kb sa[m, kb] * sw[n / 128, kb] * sum_{k in kb} a[m, k] * w[n, k]
//
// Here the entry points and the kernel of few rows: the weights stream past blocks of 16 or 32 of
// them (weight_stream.cuh); HBM is the bound.  A tile is a row block of 256 features, the row
// blocks of the same features next to one another, so that the weights come from HBM once.
// More rows: product_tiles.cu.
#include <string.h>

#include <new>

#include "product.cuh"

#define MOE_EXPORT extern "C" __attribute__((visibility("default")))

struct moe_product_s {
  moe_product_config cfg;
  size_t ws_bytes, off_counters, off_part;
  unsigned long long wait_limit_ns;
};

namespace moe {
namespace {

template <int ROWS>
struct RowsSmem {
  WsSmem<true, ROWS, ROWS, ROWS == 16 ? 6 : 5> ws;          // as many stages as 227 KB hold
};

template <int ROWS>
__global__ void __launch_bounds__(kWsBlock, 1)
    product_rows_kernel(const __grid_constant__ CUtensorMap wmap,
                        const __grid_constant__ CUtensorMap amap, const ProductArgs p) {
  extern __shared__ uint8_t smem_raw[];
  RowsSmem<ROWS>& s = *reinterpret_cast<RowsSmem<ROWS>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  using S = decltype(s.ws);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;
  const int per = p.kb;                               // stages of a tile
  const int blocks = (p.M + ROWS - 1) / ROWS, part_rows = min(p.M, ROWS);
  const WsSplit split((p.N + kWsRows - 1) / kWsRows * blocks, per, ctas);
  const int ub = split.begin(cta), ue = split.begin(cta + 1);
  const WsRole role{p.wait_limit_ns, p.status, MOE_DEV_WAIT_TIMEOUT_PRODUCT};
  ws_setup(s.ws);

  if (warp == 1) {
    WsWeights<S> out(s.ws, role, blocks > 1);
    for (int u = ub; u < ue; ++u) {
      const int tile = u / per, row = tile / blocks * kWsRows;
      out.load(&wmap, row, row + kWsBoxRows < p.N ? row + kWsBoxRows : -1,
               (u - tile * per) * kWsBytes);
    }
    out.drain();
  } else if (warp == 2) {
    WsMma<S> mma(s.ws, role);
    for (int u = ub; u < ue; ++u) mma.stage(true, true);
    mma.drain();
  } else if (warp == 3) {
    WsActivations<S> out(s.ws, role);
    // past the end of N the last block of weights, whose sums are not used
    for (int u = ub; u < ue; ++u) {
      const int tile = u / per, c = u - tile * per, f = tile / blocks, m0 = (tile - f * blocks) * ROWS;
      const float *sx = nullptr, *sw = nullptr;
      if (lane < ROWS && m0 + lane < p.M) sx = p.sa + (size_t)(m0 + lane) * p.kb + c;
      if (lane < 2) sw = p.sw + (size_t)min(2 * f + lane, (p.N - 1) / 128) * p.kb + c;
      out.load(&amap, m0, c * kWsBytes, ROWS, sx, sw);
    }
    out.drain();
  } else if (ws_is_promoter()) {
    WsPromoter<S> sum(s.ws, role);
    ws_each_run(split, per, [&](int tile, int c0, int c1, int) {
      const bool take = lane < ROWS && tile % blocks * ROWS + lane < p.M;
      sum.clear();
      for (int c = c0; c < c1; ++c) sum.add(1.f, take);
      ws_tile_free();
      sum.park(ROWS);
      ws_tile_ready();
    });
  } else {
    const int tid = ws_worker_thread();
    WsRole wait = role;
    ws_each_run(split, per, [&](int tile, int, int, int t0) {
      ws_tile_free();
      ws_tile_ready();
      const WsShare share(split, t0, per);
      const int parts = share.finishers();
      if (share.b0 != share.b1 && (cta == share.b1 || parts > 1))
        ws_store_partial(s.ws.tile, ws_partial(p.part, part_rows, cta, cta == share.b0), part_rows);
      if (share.b0 != share.b1 && cta == share.b1) return;
      // a part of the columns, four of a row a thread at a time
      const int f = tile / blocks, m0 = (tile - f * blocks) * ROWS, rows = min(ROWS, p.M - m0);
      const int mine = cta - share.b0, q0 = (kWsRows / 4) * mine / parts,
                q = (kWsRows / 4) * (mine + 1) / parts - q0;
#pragma unroll 1
      for (int i = tid; i < rows * q; i += kWsThreads) {
        const int m = i / q, col = 4 * (q0 + i - m * q), n = f * kWsRows + col;
        if (n >= p.N) continue;
        float v[4];
        ws_tile_values(s.ws.tile[m], p.part, part_rows, share, m, col, wait, v);
        store_out4(p, m0 + m, n, make_float4(v[0], v[1], v[2], v[3]));
      }
    });
  }
  ws_teardown(s.ws);
}

template <int ROWS>
cudaError_t launch_rows(const ProductArgs& a, int ctas, cudaStream_t st) {
  CUtensorMap am, wm;
  if (!ws_map(&am, a.a, a.K, a.M, ROWS) || !ws_map(&wm, a.w, a.K, a.N, kWsBoxRows))
    return cudaErrorInvalidValue;
  // the status word and, where tiles are shared, the partial tiles: heads, and tails if a tile
  // has more than two CTAs
  const int blocks = (a.M + ROWS - 1) / ROWS, part_rows = a.M < ROWS ? a.M : ROWS;
  const WsSplit split((a.N + kWsRows - 1) / kWsRows * blocks, a.kb, ctas);
  const int slots = split.whole(a.kb) ? 0 : split.each >= a.kb ? kWsCtas : 2 * kWsCtas;
  const cudaError_t e = cudaMemsetAsync(
      a.status, 0, product_head_bytes(a) + sizeof(float) * slots * part_rows * kWsRows, st);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(kWsBlock, 1, 1);
  cfg.dynamicSmemBytes = sizeof(RowsSmem<ROWS>) + 1024;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];                        // the CTAs wait for one another
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, product_rows_kernel<ROWS>, wm, am, a);
}

// Whether row blocks of 32 are quicker than 256-row tiles: a stage of the stream (256 features of a
// block against 128 K) takes a CTA 900 clocks, the meeting of the CTAs 5000 more than the end
// of a tile, and the tiles what product_tiles.cu reckons.  Replayed from a graph, as decode
// runs them: 64 rows of 4096 x 7168 16.5 us as blocks, 19.9 as tiles; 77 of 1111 x 1200 12.7
// and 18.5; 128 of 7168 x 2048 18.5 and 16.4.  Called one after another, where blocks pay their
// memset and cooperative launch in full: 20.6 and 20.6, 16.5 and 20.3, 22.6 and 16.7.  Of 75
// sizes replayed (40 to 128 rows) the rule missed the quicker form in 3, by 6 % at most.
// Units are divided by all CTAs although small work goes to fewer (WsSplit): with the units
// that these really take it missed 7, four of them by 40 to 50 %.
bool rows_are_few(const ProductArgs& p, int ctas, int num_sms) {
  if (p.M <= kProductRows) return true;
  if (p.M > kProductBlocks * kProductRows) return false;
  const long long blocks = (p.M + kProductRows - 1) / kProductRows;
  const long long units = (p.N + kWsRows - 1) / kWsRows * blocks * p.kb;
  return units < (1 << 30) && (units + ctas - 1) / ctas * 900 + 5000 < product_tiles_clocks(p, num_sms);
}

template <int ROWS>
cudaError_t prepare_rows() {
  static_assert(sizeof(RowsSmem<ROWS>) + 1024 <= 227 * 1024, "shared memory of one CTA");
  return cudaFuncSetAttribute(product_rows_kernel<ROWS>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)sizeof(RowsSmem<ROWS>) + 1024);
}

}  // namespace

cudaError_t prepare_product_kernels() {
  cudaError_t e = prepare_rows<16>();
  if (e == cudaSuccess) e = prepare_rows<32>();
  return e == cudaSuccess ? prepare_product_tiles() : e;
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
  static_assert(sizeof(unsigned int) * moe::kProductCounters <= 1024, "");
  // partial tiles: two a CTA of the weight stream, one a cluster pair of the tiles
  const size_t stream = sizeof(float) * 2 * moe::kWsCtas * moe::kWsRows *
                        (size_t)(cfg->max_rows <= 16 ? 16 : moe::kProductRows);
  const size_t tiles = sizeof(float) * moe::kProductPairs * 256 * 256;
  p->ws_bytes = p->off_part + (cfg->max_rows > moe::kProductRows && tiles > stream ? tiles : stream);
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
  moe_status s = moe::check_device(moe::KernelSet::kProduct, &sms);
  if (s != MOE_OK) return s;
  auto* st = static_cast<cudaStream_t>(stream);
  auto* ws = static_cast<uint8_t*>(workspace);
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
  g.a = static_cast<const uint8_t*>(a);
  g.sa = a_scales;
  g.out = out;
  g.M = rows;
  const int ctas = sms < moe::kWsCtas ? sms : moe::kWsCtas;
  return moe::cuda_status(rows <= 16                      ? moe::launch_rows<16>(g, ctas, st)
                          : moe::rows_are_few(g, ctas, sms) ? moe::launch_rows<32>(g, ctas, st)
                                                          : moe::launch_product_tiles(g, sms, st));
}

MOE_EXPORT moe_status moe_product_device_status(moe_product_t product, void* workspace,
                                                void* stream, uint32_t* bits) {
  if (product == nullptr || workspace == nullptr) return MOE_ERR_INVALID_ARG;
  return moe::read_device_status(static_cast<unsigned int*>(workspace),
                                 static_cast<cudaStream_t>(stream), bits);
}

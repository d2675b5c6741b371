// A whole mixture-of-experts layer for a few tokens (1..16) in one kernel.
//
//   l = x Wr^T + b;  ids = top-k;  w = softmax;  h_e = silu(Wg_e x) * (Wu_e x);
//   out[t] = bf16( sum_j w_j Wd_{ids_j} h_{ids_j} + Wd_s h_s )
//
// For a few tokens the layer is one read of the selected experts' weights: every weight
// meets at most 16 rows, so HBM bounds it, and what a chain of kernels adds to that read
// (launches, ramps and tails of each, the permutation) is what this kernel takes out.
// One cooperative launch, one CTA per SM, in three phases separated by two grid barriers:
//
//   1. router: an (expert, K split) item a CTA, fp32 dot products on the FMA units (7 MB
//      of weights at most).  FP8: x is quantised per 1x128 group here.
//   2. every CTA selects the experts of all tokens itself (a warp a token; reading T * E
//      logits from L2 is cheaper than another barrier), then gate/up over the distinct
//      experts that some token selected: a tile is 32 features, their 32 gate rows and 32
//      up rows of one expert, and multiplies all tokens at once, since a product's columns
//      are there whether used or not; only the routed ones are kept, so no permutation.
//   3. down: a tile is 64 output columns, its K axis the concatenated h of every selected
//      expert, accumulated with the routing weights; so the combine is the K loop itself,
//      and nothing is left to add up after it.
//
// Weights arrive through the ring of weight_stream.cuh, whose producer runs ahead through
// the barriers: the shared expert's gate/up rows load during the router phase, and the
// first down rows while the CTAs meet after gate/up.  h keeps fp32's precision as two bf16
// parts (bf16 weights), or is quantised per 1x128 group by the CTA that stores a group's
// last tile (FP8).  Every sum is fp32 and in an order fixed by the shapes and the routing.
#include <cudaTypedefs.h>

#include "weight_stream.cuh"

namespace moe {
namespace {

constexpr int kShared = kFewSlots;                    // slot of the shared expert
constexpr unsigned long long kDrainNs = 1000000000ull;

template <int NT>
struct FewSmem {
  static constexpr int kStages = NT == 1 ? 6 : 5;
  alignas(1024) uint8_t ring[kStages * kWsStageBytes];
  alignas(16) float red[kWsWarps * 8 * NT * kWsRedPitch];
  float w[MOE_FEW_TOKENS_MAX][kMaxTopK];              // routing weights
  int ids[MOE_FEW_TOKENS_MAX][kMaxTopK];              // routed experts, -1 in padding rows
  short active[kFewSlots];                            // the distinct experts, ascending
  signed char pick[kFewSlots + 1][MOE_FEW_TOKENS_MAX];  // j with ids[t][j] = active[slot], or -1
  unsigned int bitmap[kMaxExperts / 32];
  uint64_t full[kStages], empty[kStages], routed;
  int flag;
};

struct FewMaps {
  CUtensorMap gate_up, down, shared_gate_up, shared_down;
};

__device__ __forceinline__ void consumers_sync() { named_bar_sync(1, kWsThreads); }

__device__ __forceinline__ uint32_t two_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <bool FP8, int NT>
__global__ void __launch_bounds__(kWsBlock, 1) few_kernel(const __grid_constant__ FewMaps maps,
                                                          const FewArgs p) {
  extern __shared__ uint8_t smem_raw[];
  FewSmem<NT>& s = *reinterpret_cast<FewSmem<NT>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int kStages = FewSmem<NT>::kStages;
  constexpr int TT = 8 * NT;                          // token columns
  constexpr int EB = FP8 ? 1 : 2;                     // bytes of a weight
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;
  const int hb = p.H * EB;                            // bytes of a gate/up row
  const int ch_h = (hb + kWsBytes - 1) / kWsBytes;    // stages of a gate/up tile
  const int ch_i = (p.I * EB + kWsBytes - 1) / kWsBytes;
  const int ch_s = p.S ? (p.Is * EB + kWsBytes - 1) / kWsBytes : 0;
  const int units_s = p.S ? p.Is / 32 * ch_h : 0;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), kWsWarps);
    }
    mbar_init(smem_u32(&s.routed), 1);
    fence_mbarrier_init();
  }
  if (tid < kMaxExperts / 32) s.bitmap[tid] = 0;
  for (int i = tid; i < (kFewSlots + 1) * MOE_FEW_TOKENS_MAX; i += kWsBlock)
    (&s.pick[0][0])[i] = -1;
  __syncthreads();

  if (warp == kWsWarps) {
    // ------------------------------------------------------------------ producer
    const uint64_t once = policy_evict_first();       // weights are read once
    int stage = 0;
    uint32_t phase = 0, issued = 0, parity = 0;
    bool ok = true;
    auto load = [&](const CUtensorMap* m, int row0, int row1, int c, int row_bytes) {
      if (!ok) return;
      ok = ws_wait(smem_u32(&s.empty[stage]), phase ^ 1u, p.wait_limit_ns, p.status, p.timeout_bit);
      if (!ok) return;
      ws_load_stage(smem_u32(s.ring + stage * kWsStageBytes), m, row0, row1, c * kWsBytes,
                    min(kWsBytes, row_bytes - c * kWsBytes), smem_u32(&s.full[stage]), once);
      issued |= 1u << stage;
      parity = (parity & ~(1u << stage)) | (phase << stage);
      if (++stage == kStages) { stage = 0; phase ^= 1u; }
    };
    auto gate_up = [&](const CUtensorMap* m, int I, int units, bool routed) {
      const int ft = I / 32;
      const WsSplit split(units, ctas);
      const int u1 = split.begin(cta + 1);
      for (int u = split.begin(cta); u < u1 && ok; ++u) {
        const int tile = u / ch_h, c = u - tile * ch_h;
        const int slot = routed ? tile / ft : 0, f = (routed ? tile - slot * ft : tile) * 32;
        const int row = (routed ? s.active[slot] * 2 * I : 0) + f;
        load(m, row, row + I, c, hb);
      }
    };
    gate_up(&maps.shared_gate_up, p.Is, units_s, false);
    if (ok)
      ok = ws_wait(smem_u32(&s.routed), 0, p.wait_limit_ns, p.status, p.timeout_bit);
    if (ok) {
      int A = 0;
      for (int i = 0; i < kMaxExperts / 32; ++i) A += __popc(s.bitmap[i]);
      gate_up(&maps.gate_up, p.I, A * (p.I / 32) * ch_h, true);
      if (A > 0) {
        const int per = ch_s + A * ch_i;              // stages of a down tile
        const WsSplit split(p.H / 64 * per, ctas);
        const int u1 = split.begin(cta + 1);
        for (int u = split.begin(cta); u < u1 && ok; ++u) {
          const int tile = u / per;
          int c = u - tile * per;
          const bool shared = c < ch_s;
          int row = tile * 64;
          if (!shared) {
            const int slot = (c - ch_s) / ch_i;
            c -= ch_s + slot * ch_i;
            row += s.active[slot] * p.H;
          }
          load(shared ? &maps.shared_down : &maps.down, row, row + 32, c, (shared ? p.Is : p.I) * EB);
        }
      }
    }
    // no copy may still be writing when the CTA leaves
    for (int i = 0; i < kStages; ++i)
      if ((issued >> i) & 1u)
        ws_wait(smem_u32(&s.full[i]), (parity >> i) & 1u, kDrainNs, p.status, p.timeout_bit);
    return;
  }

  // -------------------------------------------------------------------- consumers
  const int g = lane >> 2, q = lane & 3;
  const int kb_h = p.H / 128, kb_i = p.imax / 128;
  bool ok = true;

  // all CTAs meet; what they stored before is visible after
  auto grid_sync = [&](unsigned int* counter) {
    consumers_sync();
    if (tid == 0) {
      __threadfence();
      atomicAdd(counter, 1u);
      bool met = ld_acquire_gpu(counter) >= (unsigned int)ctas;
      const uint64_t t0 = global_timer_ns();
      while (!met) {
        met = ld_acquire_gpu(counter) >= (unsigned int)ctas;
        if (!met && global_timer_ns() - t0 >= p.wait_limit_ns) {
          atomicOr(p.status, p.timeout_bit);
          break;
        }
      }
      s.flag = met;
    }
    consumers_sync();
    if (!s.flag) ok = false;
  };

  // ---- 1. router logits of all tokens, items (expert, K split)
  for (int item = cta; item < p.E * p.router_splits; item += ctas) {
    const int split = item / p.E, e = item - split * p.E;
    const int k0 = split * p.router_k, k1 = min(p.H, k0 + p.router_k);
    const float* wr = p.router_w + (size_t)e * p.H;
    float acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = 0.f;
    for (int k = k0 + warp * 256 + lane * 8; k < k1; k += kWsWarps * 256) {
      const float4 w0 = __ldg(reinterpret_cast<const float4*>(wr + k));
      const float4 w1 = __ldg(reinterpret_cast<const float4*>(wr + k + 4));
      const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
      uint4 xv[TT];                                   // columns past T repeat the last token
#pragma unroll
      for (int t = 0; t < TT; ++t)
        xv[t] = __ldg(reinterpret_cast<const uint4*>(p.x + (size_t)min(t, p.T - 1) * p.H + k));
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const uint32_t r[4] = {xv[t].x, xv[t].y, xv[t].z, xv[t].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[t] = fmaf(__uint_as_float(r[i] << 16), w[2 * i], acc[t]);
          acc[t] = fmaf(__uint_as_float(r[i] & 0xffff0000u), w[2 * i + 1], acc[t]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], off);
      if (lane == 0) s.red[warp * TT + t] = acc[t];
    }
    consumers_sync();
    if (tid < p.T) {
      float l = 0.f;
      for (int w = 0; w < kWsWarps; ++w) l += s.red[w * TT + tid];
      p.logits[((size_t)split * MOE_FEW_TOKENS_MAX + tid) * p.E + e] = l;
    }
    consumers_sync();
  }
  // counters of phases 2 and 3
  for (int i = cta * kWsThreads + tid; i < p.n_counters; i += ctas * kWsThreads) p.counters[i] = 0;
  if (FP8) {
    // x per 1x128 group, a warp a group: codes of x / s, s = amax / 448
    for (int i = cta * kWsWarps + warp; i < p.T * kb_h; i += ctas * kWsWarps) {
      const int t = i / kb_h, kb = i - t * kb_h;
      if (p.valid != nullptr && !p.valid[t]) continue;
      const uint2 v = *reinterpret_cast<const uint2*>(p.x + (size_t)t * p.H + kb * 128 + lane * 4);
      const float f[4] = {__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                          __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u)};
      float sc;
      const uint32_t codes = quantize_group_lane(f, &sc);
      *reinterpret_cast<uint32_t*>(p.xq + (size_t)t * p.H + kb * 128 + lane * 4) = codes;
      if (lane == 0) p.sx[(size_t)t * kb_h + kb] = sc;
    }
  }
  grid_sync(p.bar);

  // ---- 2a. the experts of every token, by every CTA for itself
  for (int t = warp; t < p.T; t += kWsWarps) {
    const bool real = p.valid == nullptr || p.valid[t];
    // Logits as keys of their order (larger float, larger key; -0 as +0; at least 1, and 0 once
    // taken), so that a round is two warp reductions: the largest key, then the lowest expert
    // that has it.  The rounds are a loop, not unrolled: every launch fetches this code anew,
    // and it runs once (unrolled, the selection took 11000 clocks for 8 experts, as a loop
    // 3000).
    float v[8];
    uint32_t key[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane + 32 * i;
      float part[kFewRouterSplits], bias = 0.f;       // every load before the first use
      if (e < p.E) {
        if (p.router_b != nullptr) bias = p.router_b[e];
#pragma unroll
        for (int sp = 0; sp < kFewRouterSplits; ++sp)
          if (sp < p.router_splits)
            part[sp] = __ldcg(p.logits + ((size_t)sp * MOE_FEW_TOKENS_MAX + t) * p.E + e);
      }
      v[i] = 0.f;
      key[i] = 0;
      if (e < p.E) {
#pragma unroll
        for (int sp = 0; sp < kFewRouterSplits; ++sp)
          if (sp < p.router_splits) v[i] += part[sp];
        v[i] += bias;
        const uint32_t u = __float_as_uint(v[i] + 0.f);
        key[i] = max(u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u), 1u);
        if (cta == 0 && p.logits_out != nullptr)
          p.logits_out[(size_t)t * p.E + e] = real ? v[i] : 0.f;
      }
    }
    int mine_e = -1;                                  // lane j: the j-th expert and its logit
    float mine_v = 0.f;
    if (real) {
#pragma unroll 1
      for (int j = 0; j < p.k; ++j) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) best = max(best, key[i]);
        best = __reduce_max_sync(0xffffffffu, best);
        int e = kMaxExperts;
#pragma unroll
        for (int i = 7; i >= 0; --i)
          if (key[i] == best) e = lane + 32 * i;
        e = __reduce_min_sync(0xffffffffu, e);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (e == lane + 32 * i) key[i] = 0;
        if (lane == j) {
          mine_e = e;
          mine_v = __uint_as_float(best ^ ((best >> 31) ? 0x80000000u : 0xffffffffu));
        }
      }
    }
    const float top = __shfl_sync(0xffffffffu, mine_v, 0);
    const float ex = real && lane < p.k ? expf(mine_v - top) : 0.f;
    float z = ex;
    if (!p.renorm) {
      z = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (lane + 32 * i < p.E) z += expf(v[i] - top);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
    if (lane < p.k) {
      const float w = real ? ex / z : 0.f;
      s.ids[t][lane] = mine_e;
      s.w[t][lane] = w;
      if (real) atomicOr(&s.bitmap[mine_e >> 5], 1u << (mine_e & 31));
      if (cta == 0 && p.ids_out != nullptr) p.ids_out[t * p.k + lane] = mine_e;
      if (cta == 0 && p.w_out != nullptr) p.w_out[t * p.k + lane] = w;
    }
  }
  consumers_sync();
  auto rank_of = [&](int e) {
    int r = __popc(s.bitmap[e >> 5] & ((1u << (e & 31)) - 1u));
#pragma unroll
    for (int i = 0; i < kMaxExperts / 32 - 1; ++i)
      if (i < (e >> 5)) r += __popc(s.bitmap[i]);
    return r;
  };
  if (tid < p.E && ((s.bitmap[tid >> 5] >> (tid & 31)) & 1u)) s.active[rank_of(tid)] = (short)tid;
  if (tid < p.T * p.k) {
    const int t = tid / p.k, j = tid - t * p.k, e = s.ids[t][j];
    if (e >= 0) s.pick[rank_of(e)][t] = (signed char)j;
  }
  if (tid < p.T && s.ids[tid][0] >= 0) s.pick[kShared][tid] = 0;
  int A = 0;
  for (int i = 0; i < kMaxExperts / 32; ++i) A += __popc(s.bitmap[i]);
  consumers_sync();
  if (tid == 0) mbar_arrive(smem_u32(&s.routed));

  // row of h of token t at a slot, or -1
  auto h_row = [&](int slot, int t) {
    if (t >= p.T) return -1;
    const int j = s.pick[slot][t];
    return j < 0 ? -1 : slot == kShared ? p.T * p.k + t : t * p.k + j;
  };
  int stage = 0;
  uint32_t phase = 0;
  const uint32_t lane_off = ws_lane_offset(warp, lane);
  auto stage_wait = [&]() {
    if (ok)
      ok = ws_wait(smem_u32(&s.full[stage]), phase, p.wait_limit_ns, p.status, p.timeout_bit);
  };
  auto stage_done = [&]() {
    __syncwarp();
    if (lane == 0 && ok) mbar_arrive(smem_u32(&s.empty[stage]));
    if (++stage == kStages) { stage = 0; phase ^= 1u; }
  };
  // Where several CTAs share a tile: true for the one that arrives last.  What every
  // thread stored before is visible to it after.
  auto arrive_last = [&](unsigned int* counter, unsigned int expected) {
    consumers_sync();
    if (tid == 0) {
      __threadfence();
      s.flag = atomicAdd(counter, 1u) + 1 == expected;
      __threadfence();
    }
    consumers_sync();
    return s.flag != 0;
  };
  // ---- 2b. gate/up
  auto gate_up = [&](bool routed, int I, int units, unsigned int* split_count, float* parts) {
    const int ft = I / 32;
    const WsSplit split(units, ctas);
    const uint8_t* xb = FP8 ? p.xq : reinterpret_cast<const uint8_t*>(p.x);
    const int u1 = split.begin(cta + 1);
    for (int u = split.begin(cta); u < u1;) {
      const int tile = u / ch_h, c0 = u - tile * ch_h, c1 = min(ch_h, c0 + (u1 - u)), t0 = u - c0;
      u += c1 - c0;
      const int slot = routed ? tile / ft : kShared, f = (routed ? tile - slot * ft : tile) * 32;
      const int e = routed ? s.active[slot] : 0;
      const float* sw_gate = nullptr;
      const float* sw_up = nullptr;
      if (FP8) {
        const float* sw = routed ? p.s_gate_up + (size_t)e * (2 * I / 128) * kb_h : p.ss_gate_up;
        sw_gate = sw + (size_t)(f / 128) * kb_h;
        sw_up = sw + (size_t)((I + f) / 128) * kb_h;
      }
      bool on[NT], on2[NT][2];                        // tokens of this lane's fragment, columns
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        on[n] = h_row(slot, n * 8 + g) >= 0;
        on2[n][0] = h_row(slot, n * 8 + 2 * q) >= 0;
        on2[n][1] = h_row(slot, n * 8 + 2 * q + 1) >= 0;
      }
      struct Frag {
        uint4 b[1][NT];
        float fa[NT][2], fg, fu;                      // FP8: scales of tokens, gate and up rows
      };
      auto fetch = [&](int c, Frag& x) {
        const int kbyte = c * kWsBytes + warp * 64;
        const bool live = kbyte < hb;                 // H is a multiple of 128: all or nothing
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          x.b[0][n] = make_uint4(0, 0, 0, 0);
          if (live && on[n])
            x.b[0][n] = __ldcg(reinterpret_cast<const uint4*>(xb + (size_t)(n * 8 + g) * hb +
                                                              kbyte + q * 16));
          if (FP8) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
              x.fa[n][i] = live && on2[n][i]
                               ? __ldcg(p.sx + (size_t)(n * 8 + 2 * q + i) * kb_h + kbyte / 128)
                               : 0.f;
          }
        }
        if (FP8) {
          x.fg = live ? sw_gate[kbyte / 128] : 0.f;
          x.fu = live ? sw_up[kbyte / 128] : 0.f;
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
          stage_wait();
          if (ok && (c + j) * kWsBytes + warp * 64 < hb) {
            const uint32_t slice = smem_u32(s.ring + stage * kWsStageBytes) + lane_off;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              if (FP8) {
                float part[NT][4] = {};
                ws_multiply<FP8, NT, 1>(slice, m, x[j].b, part);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                  for (int i = 0; i < 4; ++i)
                    acc[m][n][i] = fmaf(part[n][i], (m < 2 ? x[j].fg : x[j].fu) * x[j].fa[n][i & 1],
                                        acc[m][n][i]);
              } else {
                ws_multiply<FP8, NT, 1>(slice, m, x[j].b, acc[m]);
              }
            }
          }
          stage_done();
        }
      }
      ws_park<NT>(s.red, warp, lane, acc);
      consumers_sync();
      // features f + r, f + r + 1 of token t
      const int t = tid >> 4, r = (tid & 15) * 2;
      const bool mine = tid < TT * 16;
      float2 vg = make_float2(0.f, 0.f), vu = vg;
      if (mine) {
        vg = ws_sum<NT>(s.red, t, r);
        vu = ws_sum<NT>(s.red, t, 32 + r);
      }
      bool finish = true;
      if (c1 - c0 < ch_h) {
        const int b0 = split.owner(t0), b1 = split.owner(t0 + ch_h - 1);
        if (mine) {
          float* o = ws_partial(parts, cta, b0) + t * kWsRows + r;
          *reinterpret_cast<float2*>(o) = vg;
          *reinterpret_cast<float2*>(o + 32) = vu;
        }
        finish = arrive_last(split_count + b0, b1 - b0 + 1);
        if (finish && mine) {
          vg = ws_joined(parts, b0, b1, t, r);
          vu = ws_joined(parts, b0, b1, t, 32 + r);
        }
      }
      if (finish) {
        const int row = mine ? h_row(slot, t) : -1;
        if (row >= 0) {
          const float a = vg.x / (1.0f + expf(-vg.x)) * vu.x;
          const float b2 = vg.y / (1.0f + expf(-vg.y)) * vu.y;
          if (FP8) {
            *reinterpret_cast<float2*>(p.h32 + (size_t)row * p.imax + f + r) = make_float2(a, b2);
          } else {
            // h = high + low, each the nearest bf16 of what is left: 16 bits of fraction
            const uint32_t hi = two_bf16(a, b2);
            const uint32_t lo = two_bf16(a - __uint_as_float(hi << 16),
                                         b2 - __uint_as_float(hi & 0xffff0000u));
            uint8_t* o = p.h + ((size_t)row * 2 * p.imax + f + r) * 2;
            *reinterpret_cast<uint32_t*>(o) = hi;
            *reinterpret_cast<uint32_t*>(o + (size_t)p.imax * 2) = lo;
          }
        }
        if (FP8 && arrive_last(p.group_count + (size_t)(routed ? slot + p.S : 0) * kb_i + f / 128,
                               128 / 32)) {
          // the four tiles of this 1x128 group are stored: quantise it
          for (int tt = warp; tt < p.T; tt += kWsWarps) {
            const int hr = h_row(slot, tt);
            if (hr < 0) continue;
            const float4 v = __ldcg(reinterpret_cast<const float4*>(
                p.h32 + (size_t)hr * p.imax + (f & ~127) + lane * 4));
            const float fv[4] = {v.x, v.y, v.z, v.w};
            float sc;
            const uint32_t codes = quantize_group_lane(fv, &sc);
            *reinterpret_cast<uint32_t*>(p.h + (size_t)hr * p.imax + (f & ~127) + lane * 4) = codes;
            if (lane == 0) p.sh[(size_t)hr * kb_i + f / 128] = sc;
          }
        }
      }
      consumers_sync();                               // red and flag are free again
    }
  };
  if (A > 0) {
    if (p.S) gate_up(false, p.Is, units_s, p.split_count, p.part);
    gate_up(true, p.I, A * (p.I / 32) * ch_h, p.split_count + kFewMaxCtas,
            p.part + kFewMaxCtas * 2 * kWsTileFloats);
  } else {
    // every row is padding: nothing is computed, the shared rows that were loaded are let go
    const WsSplit split(units_s, ctas);
    for (int u = split.begin(cta); u < split.begin(cta + 1); ++u) {
      stage_wait();
      stage_done();
    }
  }
  grid_sync(p.bar + 1);

  // ---- 3. down and combine
  if (A == 0) {
    const int n = p.T * p.H / 8;
    for (int i = cta * kWsThreads + tid; i < n; i += ctas * kWsThreads)
      reinterpret_cast<uint4*>(p.out)[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  const int per = ch_s + A * ch_i;
  const WsSplit down(p.H / 64 * per, ctas);
  const int u1 = down.begin(cta + 1);
  constexpr int PARTS = FP8 ? 1 : 2;
  for (int u = down.begin(cta); u < u1;) {
    const int tile = u / per, c0 = u - tile * per, c1 = min(per, c0 + (u1 - u)), t0 = u - c0;
    u += c1 - c0;
    // stage c of the tile: activation fragments, the factor of each token column, and which
    // of the columns take part
    struct Frag {
      uint4 b[PARTS][NT];
      float fh[NT][2], fw;                            // FP8: scales of h and of the weights
      int slot;                                       // -1: past the segment's K
    };
    auto fetch = [&](int c, Frag& x) {
      int slot = kShared, ci = c, width = p.Is;
      if (c >= ch_s) {
        slot = (c - ch_s) / ch_i;
        ci = c - ch_s - slot * ch_i;
        width = p.I;
      }
      const int kbyte = ci * kWsBytes + warp * 64;
      const bool live = kbyte < width * EB;
      x.slot = live ? slot : -1;
      x.fw = 1.f;
      if (FP8 && live) {
        const int rb = tile * 64 / 128, kbs = width / 128;
        x.fw = slot == kShared
                 ? p.ss_down[(size_t)rb * kbs + kbyte / 128]
                 : p.s_down[((size_t)s.active[slot] * kb_h + rb) * kbs + kbyte / 128];
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int row = live ? h_row(slot, n * 8 + g) : -1;
#pragma unroll
        for (int w = 0; w < PARTS; ++w) {
          x.b[w][n] = make_uint4(0, 0, 0, 0);
          if (row >= 0)
            x.b[w][n] = __ldcg(reinterpret_cast<const uint4*>(
                p.h + ((size_t)row * PARTS + w) * p.imax * EB + kbyte + q * 16));
        }
        if (FP8) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int hr = live ? h_row(slot, n * 8 + 2 * q + i) : -1;
            x.fh[n][i] = hr >= 0 ? __ldcg(p.sh + (size_t)hr * kb_i + kbyte / 128) : 0.f;
          }
        }
      }
    };
    float acc[4][NT][4];
    ws_zero<NT>(acc);
    Frag x[3];
    fetch(c0, x[0]);
    if (c0 + 1 < c1) fetch(c0 + 1, x[1]);
    for (int c = c0; c < c1; c += 3) {
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        if (c + j >= c1) break;
        if (c + j + 2 < c1) fetch(c + j + 2, x[(j + 2) % 3]);
        stage_wait();
        if (ok && x[j].slot >= 0) {
          // the factor of each token column, and which columns take part
          float f[NT][2];
          uint32_t keep = 0;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int t = n * 8 + 2 * q + i, pick = s.pick[x[j].slot][t];
              if (pick >= 0) keep |= 1u << (2 * n + i);
              f[n][i] = x[j].slot == kShared || pick < 0 ? 1.f : s.w[t][pick];
              if (FP8) f[n][i] *= x[j].fw * x[j].fh[n][i];
            }
          const uint32_t slice = smem_u32(s.ring + stage * kWsStageBytes) + lane_off;
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            float part[NT][4] = {};
            ws_multiply<FP8, NT, PARTS>(slice, m, x[j].b, part);
            // a token that did not select this expert takes nothing from it, not even 0 * inf
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if ((keep >> (2 * n + (i & 1))) & 1u)
                  acc[m][n][i] = fmaf(part[n][i], f[n][i & 1], acc[m][n][i]);
          }
        }
        stage_done();
      }
    }
    ws_park<NT>(s.red, warp, lane, acc);
    consumers_sync();
    bool finish = true;
    const bool split = c1 - c0 < per;
    const int b0 = down.owner(t0), b1 = down.owner(t0 + per - 1);
    if (split) {
      for (int i = tid; i < TT * 32; i += kWsThreads) {
        const int t = i >> 5, r = (i & 31) * 2;
        *reinterpret_cast<float2*>(ws_partial(p.part, cta, b0) + t * kWsRows + r) =
            ws_sum<NT>(s.red, t, r);
      }
      finish = arrive_last(p.split_count + 2 * kFewMaxCtas + b0, b1 - b0 + 1);
    }
    if (finish) {
      for (int i = tid; i < TT * 32; i += kWsThreads) {
        const int t = i >> 5, r = (i & 31) * 2;
        if (t >= p.T) continue;
        const float2 v = split ? ws_joined(p.part, b0, b1, t, r) : ws_sum<NT>(s.red, t, r);
        *reinterpret_cast<uint32_t*>(p.out + (size_t)t * p.H + tile * 64 + r) =
            s.ids[t][0] >= 0 ? two_bf16(v.x, v.y) : 0u;
      }
    }
    consumers_sync();                                 // red and flag are free again
  }
}

template <bool FP8, int NT>
cudaError_t launch(const FewMaps& m, const FewArgs& a, int ctas, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(kWsBlock, 1, 1);
  cfg.dynamicSmemBytes = sizeof(FewSmem<NT>) + 1024;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];                        // the CTAs wait for one another
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few_kernel<FP8, NT>, m, a);
}

template <bool FP8, int NT>
cudaError_t prepare() {
  static_assert(sizeof(FewSmem<NT>) + 1024 <= 227 * 1024, "shared memory of one CTA");
  return cudaFuncSetAttribute(few_kernel<FP8, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)sizeof(FewSmem<NT>) + 1024);
}

}  // namespace

bool ws_weight_map(CUtensorMap* m, const void* w, uint64_t row_bytes, uint64_t rows) {
  static const auto encode = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  if (encode == nullptr) return false;
  const cuuint64_t dims[2] = {row_bytes, rows};
  const cuuint64_t strides[1] = {row_bytes};
  const cuuint32_t box[2] = {128, kWsBoxRows};
  const cuuint32_t estr[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(w), dims, strides, box,
                estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t prepare_few_kernels() {
  cudaError_t e = prepare<false, 1>();
  if (e == cudaSuccess) e = prepare<false, 2>();
  if (e == cudaSuccess) e = prepare<true, 1>();
  if (e == cudaSuccess) e = prepare<true, 2>();
  return e;
}

cudaError_t launch_few(FewArgs a, bool fp8, int num_sms, cudaStream_t st) {
  const int ctas = num_sms < kFewMaxCtas ? num_sms : kFewMaxCtas;
  // with fewer experts than CTAs the dot products are cut along K too
  int splits = ctas / a.E;
  splits = splits < 1 ? 1 : splits > kFewRouterSplits ? kFewRouterSplits : splits;
  a.router_k = ((a.H + splits - 1) / splits + 255) / 256 * 256;
  a.router_splits = (a.H + a.router_k - 1) / a.router_k;
  const uint64_t eb = fp8 ? 1 : 2, E = a.E, H = a.H, I = a.I, Is = a.Is;
  FewMaps m;
  if (!ws_weight_map(&m.gate_up, a.w_gate_up, H * eb, E * 2 * I) ||
      !ws_weight_map(&m.down, a.w_down, I * eb, E * H))
    return cudaErrorInvalidValue;
  if (a.S == 0) {
    m.shared_gate_up = m.gate_up;      // not used
    m.shared_down = m.down;
  } else if (!ws_weight_map(&m.shared_gate_up, a.ws_gate_up, H * eb, 2 * Is) ||
             !ws_weight_map(&m.shared_down, a.ws_down, Is * eb, H)) {
    return cudaErrorInvalidValue;
  }
  if (fp8) return a.T <= 8 ? launch<true, 1>(m, a, ctas, st) : launch<true, 2>(m, a, ctas, st);
  return a.T <= 8 ? launch<false, 1>(m, a, ctas, st) : launch<false, 2>(m, a, ctas, st);
}

}  // namespace moe
